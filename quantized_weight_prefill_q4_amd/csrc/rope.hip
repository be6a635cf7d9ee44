// Rotary positions of activation rows: every head's first n_rot elements turned
// pair by pair by the row's position, the rest copied (rotary.h has the
// arithmetic).
//
// The operator moves bytes: each element is read and written once against 1.5
// operations.  What could cost more is the angles (some 40 f64 operations per
// pair), so a workgroup computes its row's once, into LDS, and all heads read them
// there.  2048 rows of 40 heads of 128, half rotated, f32: 18.4 us, 4.6 TB/s; 8192
// rows of 32 heads, f16: 22.6 us, 5.9 TB/s.  (Four rows per workgroup: 2048 rows of 32
// heads 8.9 us against 7.4.)
#include "rotary.h"

namespace mq {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    const void *x;
    void *y;
    const int32_t *pos;
    const double *freqs;
    int64_t ldx, ldy;
    int M, heads, head_dim, n_rot, x_type, y_type, interleaved, in_place;
    float mscale;
    int parts;       // workgroups that share a row's heads
    int64_t first;   // row of the launch
};

__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    extern __shared__ float2 cs[];   // [np]
    const int64_t row = a.first + blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts, position = a.pos[row];
    const HeadItems h = head_items(a.head_dim, a.n_rot, a.in_place);
    for (int j = threadIdx.x; j < h.np; j += kRopeThreads)
        cs[j] = rotation(position, a.freqs[j], a.mscale);
    __syncthreads();
    const int per_head = h.rot + h.copy, items = per_head * a.heads;
    for (int i = part * kRopeThreads + threadIdx.x; i < items; i += a.parts * kRopeThreads) {
        const int head = i / per_head, item = i - head * per_head;
        const int64_t e = (int64_t)head * a.head_dim;
        rotate_item(item, h, a.head_dim, a.interleaved, cs, a.x, a.x_type, row * a.ldx + e, a.y,
                    a.y_type, row * a.ldy + e);
    }
}

}  // namespace

hipError_t launch_rope(const RopeSpec &s, hipStream_t stream) {
    RopeArgs a;
    a.x = s.x;
    a.y = s.y;
    a.pos = s.pos;
    a.freqs = s.freqs;
    a.ldx = s.ldx;
    a.ldy = s.ldy;
    a.M = s.M;
    a.heads = s.heads;
    a.head_dim = s.head_dim;
    a.n_rot = s.n_rot;
    a.x_type = s.x_type;
    a.y_type = s.y_type;
    a.interleaved = s.interleaved;
    a.in_place = s.x == s.y;
    a.mscale = s.mscale;
    const HeadItems h = head_items(a.head_dim, a.n_rot, a.in_place);
    const int64_t items = (int64_t)(h.rot + h.copy) * a.heads;
    // a few rows are spread over workgroups, which all compute the row's angles: with many
    // rows those are work (2048 rows of 40 heads 25.6 us with two workgroups a row, 19.3
    // with one), one row of 32 heads is alone with its round trip to memory
    int64_t parts = s.M >= 512 ? 1 : (items + kRopeThreads - 1) / kRopeThreads;
    if (parts > 16) parts = 16;
    if (parts < 1) parts = 1;
    a.parts = (int)parts;
    constexpr int kMost = 1 << 23;   // rows of a launch (of fewer than 2^32 threads)
    for (a.first = 0; a.first < s.M; a.first += kMost) {
        const int64_t rows = s.M - a.first < kMost ? s.M - a.first : kMost;
        hipLaunchKernelGGL(rope_kernel, dim3((unsigned)(rows * parts)), dim3(kRopeThreads),
                           sizeof(float2) * h.np, stream, a);
    }
    return hipGetLastError();
}

}  // namespace mq
