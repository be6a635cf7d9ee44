// Rotary positions of activation rows: every head's first n_rot elements turned
// pair by pair by the row's position, the rest copied (rotary.h has the
// arithmetic).
//
// The operator moves bytes: each element is read and written once against 1.5
// operations.  What could cost more is the angles (some 40 f64 operations per
// pair), so a workgroup computes each row's once, into LDS, and all its heads
// read them there.
#include "rotary.h"

namespace mq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;   // rows of a workgroup when there are many

struct RopeArgs {
    const void *x;
    void *y;
    const int32_t *pos;
    const double *freqs;
    int64_t ldx, ldy;
    int M, heads, head_dim, n_rot, x_type, y_type, interleaved, in_place;
    float mscale;
    int parts;   // workgroups that share a group of rows' heads
};

template <int ROWS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    extern __shared__ float2 cs[];   // [ROWS][np]
    const int64_t first = (int64_t)(blockIdx.x / a.parts) * ROWS;
    const int part = blockIdx.x % a.parts;
    const int rows = (int)((a.M - first) < ROWS ? a.M - first : ROWS);
    const HeadItems h = head_items(a.head_dim, a.n_rot, a.in_place);
    for (int i = threadIdx.x; i < rows * h.np; i += kRopeThreads) {
        const int r = i / h.np, j = i - r * h.np;
        cs[i] = rotation(a.pos[first + r], a.freqs[j], a.mscale);
    }
    __syncthreads();
    const int per_head = h.rot + h.copy, per_row = per_head * a.heads;
    if (per_row == 0) return;
    for (int i = part * kRopeThreads + threadIdx.x; i < rows * per_row;
         i += a.parts * kRopeThreads) {
        const int r = i / per_row, k = i - r * per_row;
        const int head = k / per_head, item = k - head * per_head;
        const int64_t e = (int64_t)head * a.head_dim, row = first + r;
        rotate_item(item, h, a.head_dim, a.interleaved, cs + r * h.np, a.x, a.x_type,
                    row * a.ldx + e, a.y, a.y_type, row * a.ldy + e);
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
    // Several rows share a workgroup once there are enough rows for every compute
    // unit; a few rows are spread over workgroups instead.
    const bool many = s.M >= 1024;
    const int rows = many ? kRopeRows : 1;
    int64_t parts = many ? 1 : (items + kRopeThreads - 1) / kRopeThreads;
    if (parts > 16) parts = 16;
    if (parts < 1) parts = 1;
    a.parts = (int)parts;
    const int64_t groups = ((int64_t)s.M + rows - 1) / rows;
    const size_t lds = sizeof(float2) * rows * h.np;
    const dim3 grid((unsigned)(groups * parts));
    if (many)
        hipLaunchKernelGGL((rope_kernel<kRopeRows>), grid, dim3(kRopeThreads), lds, stream, a);
    else
        hipLaunchKernelGGL((rope_kernel<1>), grid, dim3(kRopeThreads), lds, stream, a);
    return hipGetLastError();
}

}  // namespace mq
