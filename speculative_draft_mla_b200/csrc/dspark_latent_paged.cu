// Attention of new tokens over the paged latent cache: dispatch.
#include "dspark_latent.cuh"

namespace dspark {

cudaError_t launch_paged_simt(const Paged &p, cudaStream_t st);

namespace {

// Clears the error word, then sets the page bit for what only the device can
// see: sequence bounds and the pages that the sequences' keys lie in.
__global__ void k_paged_check(const Paged p) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    bool mine = false;
    for (int s = threadIdx.x >> 5; s < p.n_seq; s += blockDim.x >> 5) {
        const SeqView v = seq_view(p, s);
        mine |= v.bad;
        if (v.q_len == 0) continue;
        // the pages some row of the sequence reads
        int lo, hi, l1, h1;
        seq_range(p, v, 0, &lo, &h1);
        seq_range(p, v, v.q_len - 1, &l1, &hi);
        if (hi <= lo) continue;
        for (int g = lo / p.page_size + (threadIdx.x & 31); g <= (hi - 1) / p.page_size; g += 32) {
            const int page = p.table[(size_t)s * p.max_pages + g];
            mine |= page < 0 || page >= p.n_pages;
        }
    }
    if (mine) bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) *p.err = bad ? kErrPage : 0u;
}

}  // namespace

size_t paged_workspace_size(const Paged &p) { return 256; }

cudaError_t launch_paged(const Paged &pp, void *ws, cudaStream_t st) {
    Paged p = pp;
    p.err = (uint32_t *)ws;
    count_launch();
    k_paged_check<<<1, 1024, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.T == 0 || p.n_seq == 0) return e;
    return launch_paged_simt(p, st);
}

}  // namespace dspark
