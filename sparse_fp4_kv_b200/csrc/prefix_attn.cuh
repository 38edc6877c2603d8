// prefix_attn.cuh -- decode attention for sequences that share a prefix.
//
// Sequences come in groups; entries below a group's prefix length are read
// through the pages of the group's first member, later ones through the
// sequence's own pages, and each query's window rows are attended too:
//     o_h = sum_j softmax_j(scale * <q_h, v_j>) v_j
// over the entries below the query's limit and its window rows (each row is
// key and value, as in attn_decode.cuh).
#pragma once

#include "common.cuh"

namespace csa2 {

struct PrefixParams {
    const uint16_t *q;  // bf16 [nq][h][512]
    csa2_kv_desc kv;
    const int32_t *members, *group_begin, *prefix_len;
    const int32_t *q_limit;  // nullable
    const uint8_t *swa;      // nullable, with begin / end
    int64_t swa_seq_stride;
    const int32_t *swa_begin, *swa_end;
    uint16_t *o;
    float *lse;        // nullable
    float scale_log2;  // softmax scale * log2(e)
    int32_t nq, q_per_seq, h, w_max, n_members, n_groups;
};

constexpr int kPsThreads = 256;
constexpr int kPsTile = 16;   // rows of a tile
constexpr int kPsHeads = 16;  // heads of a block

// One block per (member, query of the member, 16 heads); rows are staged as
// f32, a warp takes two heads' scores and statistics, a thread two columns of
// all 16 heads' outputs.
__global__ void __launch_bounds__(kPsThreads) k_prefix_attn_simple(PrefixParams p) {
    extern __shared__ float ps_smem[];
    float *qs = ps_smem;                       // [16][512]
    float *vs = qs + kPsHeads * CSA2_D;        // [kPsTile][512]
    float *sc = vs + kPsTile * CSA2_D;         // [16][kPsTile] scores, then probabilities
    float *mx = sc + kPsHeads * kPsTile;       // [16]
    float *al = mx + kPsHeads;                 // [16]
    float *ls = al + kPsHeads;                 // [16]
    int32_t *bad = reinterpret_cast<int32_t *>(ls + kPsHeads);  // [kPsTile]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int hc = (p.h + kPsHeads - 1) / kPsHeads;
    const int32_t j = blockIdx.x, qi = blockIdx.y / hc, h0 = (blockIdx.y % hc) * kPsHeads;
    const int32_t seq = p.members[j];
    int32_t g = -1;
    for (int32_t x = 0; x < p.n_groups; ++x)
        if (p.group_begin[x] <= j && j < p.group_begin[x + 1]) g = x;
    const int64_t u = (int64_t)seq * p.q_per_seq + qi;
    if (seq < 0 || seq >= p.kv.batch || g < 0 || p.group_begin[g] < 0 || p.group_begin[g + 1] > p.n_members) {
        if (tid == 0) set_error(CSA2_DEVERR_BAD_ROW);
        return;
    }
    if (u >= p.nq) return;
    const int32_t first = p.members[p.group_begin[g]];
    const int32_t prefix = max(0, p.prefix_len[g]);
    const int64_t limit = max(0, p.q_limit ? p.q_limit[u] : p.kv.seq_len[seq]);
    int32_t wb = p.swa_begin ? p.swa_begin[u] : 0, nw = p.swa_begin ? max(0, p.swa_end[u] - wb) : 0;
    if (nw > 0 && (wb < 0 || wb >= p.swa_seq_stride || nw > p.swa_seq_stride || nw > p.w_max)) {
        if (tid == 0) set_error(CSA2_DEVERR_BAD_ROW);
        nw = 0;
    }
    for (int i = tid; i < kPsHeads * CSA2_D; i += kPsThreads) {
        const int hh = h0 + i / CSA2_D;
        qs[i] = hh < p.h ? __uint_as_float((uint32_t)p.q[(u * p.h + hh) * CSA2_D + i % CSA2_D] << 16) * p.scale_log2 : 0.0f;
    }
    if (tid < kPsHeads) mx[tid] = -INFINITY, ls[tid] = 0.0f;
    float acc[kPsHeads][2];
#pragma unroll
    for (int h = 0; h < kPsHeads; ++h) acc[h][0] = acc[h][1] = 0.0f;
    const int64_t rows = limit + nw;
    for (int64_t r0 = 0; r0 < rows; r0 += kPsTile) {
        __syncthreads();
        for (int i = tid; i < kPsTile * (CSA2_D / 16); i += kPsThreads) {
            const int e = i / (CSA2_D / 16), blk = i % (CSA2_D / 16);
            const int64_t r = r0 + e;
            float *dst = vs + e * CSA2_D + blk * 16;
            int ok = 0;
            if (r < limit) {
                const int32_t holder = r < prefix ? first : seq;
                const int64_t row = holder >= 0 && holder < p.kv.batch ? physical_row(p.kv, holder, r) : -1;
                if (row >= 0) {
                    ok = 1;
                    const uint2 c = *reinterpret_cast<const uint2 *>(p.kv.codes + row * (CSA2_D / 2) + blk * 8);
                    const uint32_t sb = p.kv.scales[row * (CSA2_D / CSA2_BLOCK) + blk];
                    const float s = e4m3x2_to_float2((uint16_t)sb).x;
                    uint32_t h2[8];
                    e2m1x8_to_f16x8(c.x, *reinterpret_cast<uint32_t(*)[4]>(h2));
                    e2m1x8_to_f16x8(c.y, *reinterpret_cast<uint32_t(*)[4]>(h2 + 4));
                    for (int t = 0; t < 8; ++t) {
                        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(h2 + t));
                        dst[2 * t] = f.x * s, dst[2 * t + 1] = f.y * s;
                    }
                } else {
                    set_error(CSA2_DEVERR_BAD_ROW);
                }
            } else if (r < rows) {
                ok = 1;
                const int64_t sl = (wb + (r - limit)) % p.swa_seq_stride;
                const uint8_t *w = p.swa + ((int64_t)seq * p.swa_seq_stride + sl) * CSA2_D + blk * 16;
                for (int t = 0; t < 16; ++t) dst[t] = e4m3x2_to_float2((uint16_t)w[t]).x;
            }
            if (!ok)
                for (int t = 0; t < 16; ++t) dst[t] = 0.0f;
            if (blk == 0) bad[e] = !ok;
        }
        __syncthreads();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int h = warp * 2 + hh;
            float top = -INFINITY;
            for (int e = 0; e < kPsTile; ++e) {
                float d = 0.0f;
                for (int c = lane; c < CSA2_D; c += 32) d = fmaf(qs[h * CSA2_D + c], vs[e * CSA2_D + c], d);
#pragma unroll
                for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
                if (bad[e]) d = -INFINITY;
                if (lane == e) sc[h * kPsTile + e] = d;
                top = fmaxf(top, d);
            }
            __syncwarp();
            const float mo = mx[h], mn = fmaxf(mo, top);
            const float at = mn == -INFINITY ? 0.0f : mn;
            float pr = lane < kPsTile ? exp2f(sc[h * kPsTile + lane] - at) : 0.0f;
            if (lane < kPsTile) sc[h * kPsTile + lane] = pr;
#pragma unroll
            for (int o = 16; o; o >>= 1) pr += __shfl_xor_sync(0xFFFFFFFFu, pr, o);
            __syncwarp();
            if (lane == 0) {
                al[h] = exp2f(mo - at);
                ls[h] = ls[h] * al[h] + pr;
                mx[h] = mn;
            }
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kPsHeads; ++h) {
            acc[h][0] *= al[h], acc[h][1] *= al[h];
#pragma unroll
            for (int e = 0; e < kPsTile; ++e) {
                const float pr = sc[h * kPsTile + e];
                acc[h][0] = fmaf(pr, vs[e * CSA2_D + tid], acc[h][0]);
                acc[h][1] = fmaf(pr, vs[e * CSA2_D + tid + kPsThreads], acc[h][1]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kPsHeads; ++h) {
        if (h0 + h >= p.h) break;
        const float inv = ls[h] > 0.0f ? 1.0f / ls[h] : 0.0f;
        uint16_t *dst = p.o + (u * p.h + h0 + h) * CSA2_D;
        dst[tid] = f32_to_bf16_bits(acc[h][0] * inv);
        dst[tid + kPsThreads] = f32_to_bf16_bits(acc[h][1] * inv);
        if (tid == 0 && p.lse)
            p.lse[u * p.h + h0 + h] = ls[h] > 0.0f ? (mx[h] + log2f(ls[h])) * 0.69314718055994531f : -INFINITY;
    }
}

}  // namespace csa2
