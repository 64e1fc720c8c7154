// short_wait_probe.cu: a test-only kernel for the bounded wait of a whole warp, as the long chunks' attention over an 8-bit cache
// makes it (pa::chunk::short_wait from csrc/chunk_common.cuh).
//
// Like wait_probe.cu: built by the tests into its own shared library, never launched by a product call, with no TMA, bulk copy
// or MMA in flight when it gives up.
#ifndef PA_TEST_HOOKS
#error "short_wait_probe.cu is test infrastructure: build it with -DPA_TEST_HOOKS"
#endif

#include "../../paged_kv_cache_83_gb300/csrc/chunk_common.cuh"

namespace {

// One warp. An mbarrier expecting one arrival; with `arrive` lane 0 arrives and the wait returns at once, without it nothing
// ever arrives: the wait gives up after its limit, or with `abort` as soon as it sees that another role gave up.
__global__ void short_wait_probe_kernel(int32_t *err, int arrive, int abort, unsigned long long *elapsed_ns) {
    __shared__ alignas(8) unsigned long long bar;
    __shared__ int flag;
    const uint32_t b = pa::smem_addr(&bar);
    if (threadIdx.x == 0) {
        pa::mbar_init(b, 1);
        pa::fence_mbar_init();
        flag = abort;
    }
    __syncwarp();
    if (arrive && threadIdx.x == 0) pa::mbar_arrive(b);
    __syncwarp();
    const uint64_t t0 = pa::globaltimer_ns();
    const bool ok = pa::chunk::short_wait(b, 0, &flag);
    const unsigned same = __match_any_sync(0xffffffffu, ok);
    if (threadIdx.x == 0) {
        *elapsed_ns = pa::globaltimer_ns() - t0;
        if (!ok) pa::chunk::give_up(err, &flag);
        if (same != 0xffffffffu) pa::raise_err(err, 1 << 20);  // the lanes do not agree
    }
}

}  // namespace

extern "C" int pa_test_short_wait_probe(int32_t *err, int arrive, int abort, unsigned long long *elapsed_ns, cudaStream_t stream) {
    short_wait_probe_kernel<<<1, 32, 0, stream>>>(err, arrive, abort, elapsed_ns);
    return static_cast<int>(cudaGetLastError());
}
