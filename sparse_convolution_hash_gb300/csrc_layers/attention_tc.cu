// attention_tc.cu -- the forward pass of attention over segments on the 5th-generation tensor cores.
//
// A block keeps TILES tiles of 128 query rows (the positions of a segment, and the query heads that share a key head
// beside one another, so that keys are read once for all of them) and walks over the segment's keys 128 at a time:
//   warp 0 loads the queries once and keys and values in turn into a ring of stages (TMA);
//   warp 1 issues S = Q K^T into tensor memory and O += P V with P from tensor memory;
//   four warps for each tile take S, a thread to a row: running maximum, exponentials, P as 16 bits in the place of S.
// With two tiles the products of one run while the other's exponentials are taken.  O stays in tensor memory; it is
// rescaled only when a row's maximum has grown by more than 2^8, so almost never after the first tiles
// (sums and P carry the same factor, which the end divides out).
//
// Every wait is bounded by the library's wait limit; one that runs out sets SPC_ERR_TIMEOUT, and each role then
// waits (bounded) for what it has in flight itself before the block frees its tensor memory and returns.
#include "attention_tc.cuh"

namespace spc {

namespace {

constexpr int kKeys = 128;       // keys of a tile
constexpr float kLazy = 8.f;     // a maximum may grow by this much (log2) before sums are rescaled

template <int D, int TILES>
struct Shape {
    static constexpr int kBoxes = D / 64;
    static constexpr int kTile = 128 * 128 * kBoxes;          // bytes of 128 rows
    static constexpr int kStages = TILES == 2 ? (D == 128 ? 4 : 8) : (D == 128 ? 2 : 5);
    static constexpr int kThreads = 64 + 128 * TILES;
    static constexpr int kCols = TILES == 2 ? 512 : 256;      // tensor memory
    static constexpr int kBars = 2 * kStages + 2 + 3 * TILES;
    static constexpr size_t kSmem = 1024 + (size_t)(TILES + kStages) * kTile + 8 * kBars + 16;
};

struct Packing {
    int heads;      // query heads of a tile
    int positions;  // positions of a tile
};

template <typename T, int D, int TILES>
__global__ void __launch_bounds__(Shape<D, TILES>::kThreads, TILES == 1 ? 2 : 1)
k_attn_tc(AttnArgs a, Packing pk, uint64_t wait_ns, const __grid_constant__ CUtensorMap map_q,
          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using S = Shape<D, TILES>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* ring = smem + TILES * S::kTile;
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)S::kStages * S::kTile);
    uint64_t* empty = full + S::kStages;
    uint64_t* q_full = empty + S::kStages;
    uint64_t* drain = q_full + 1;
    uint64_t* s_full = drain + 1;
    uint64_t* p_full = s_full + TILES;
    uint64_t* o_full = p_full + TILES;
    uint32_t* s_ctrl = reinterpret_cast<uint32_t*>(o_full + TILES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    wait_for_kernel_before();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        attn_check(a.seg_q, a.segments, a.nq, a.status, tid, S::kThreads);
        if (a.seg_k != a.seg_q) attn_check(a.seg_k, a.segments, a.nk, a.status, tid, S::kThreads);
    }
    AttnTile t;
    if (!attn_tile(a.seg_q, a.seg_k, a.segments, a.nq, a.nk, TILES * pk.positions, blockIdx.x, t)) return;
    const int per = a.hq / a.hk, packs = per / pk.heads;
    const int kv = blockIdx.y / packs, head0 = kv * per + blockIdx.y % packs * pk.heads;
    int64_t lo, hi;
    attn_share(t.lo, t.hi, kKeys, blockIdx.z, a.splits, lo, hi);
    const int tiles = TILES == 2 && t.row + pk.positions < t.end ? 2 : 1;
    const int n = (int)((hi - lo + kKeys - 1) / kKeys);

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < TILES; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_full[i], 4);
            ptx::mbar_init(&o_full[i], 1);
        }
        ptx::mbar_init_fence();
    }
    if (warp == 1) {
        ptx::tmem_alloc(s_ctrl, S::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_ctrl[0];
    const uint32_t q_base = ptx::smem_u32(smem), ring_base = ptx::smem_u32(ring);
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0 && n > 0) {
            const uint32_t bytes = (uint32_t)pk.heads * pk.positions * 128;
            ptx::mbar_arrive_expect_tx(q_full, bytes * S::kBoxes * tiles);
            for (int i = 0; i < tiles; ++i)
                for (int b = 0; b < S::kBoxes; ++b)
                    ptx::tma_load3d<1>(q_base + i * S::kTile + b * 16384, &map_q, b * 64, head0, (int32_t)(t.row + i * pk.positions),
                                       ptx::smem_u32(q_full));
            int it = 0;
            for (int j = 0; j < 2 * n && ok; ++j, ++it) {
                const int s = it % S::kStages;
                if (it >= S::kStages) ok = ptx::mbar_wait(&empty[s], (it / S::kStages - 1) & 1, wait_ns);
                if (!ok) break;
                ptx::mbar_arrive_expect_tx(&full[s], S::kTile);
                for (int b = 0; b < S::kBoxes; ++b)
                    ptx::tma_load3d<1>(ring_base + s * S::kTile + b * 16384, j & 1 ? &map_v : &map_k, b * 64, kv,
                                       (int32_t)(lo + (int64_t)(j >> 1) * kKeys), ptx::smem_u32(&full[s]));
            }
            if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
            // what is in flight has to land before the block's shared memory goes
            ptx::mbar_wait(q_full, 0, kAttnDrainNs);
            for (int j = it > S::kStages ? it - S::kStages : 0; j < it; ++j)
                ptx::mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1, kAttnDrainNs);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMAs
        if (lane == 0 && n > 0) {
            const int steps = (a.d + 15) / 16;
            const uint32_t id_s = ptx::idesc_make(AttnFmt<T>::v, 128, kKeys);
            const uint32_t id_o = ptx::idesc_make(AttnFmt<T>::v, 128, steps * 16) | 1u << 16;
            auto stage = [&](int it) { return ring_base + (uint32_t)(it % S::kStages) * S::kTile; };
            auto arrived = [&](int it) { return ptx::mbar_wait(&full[it % S::kStages], (it / S::kStages) & 1, wait_ns); };
            auto scores = [&](int i, int j) {
                attn_mma_ss(tmem + i * 128, q_base + i * S::kTile, 16384, stage(2 * j), 16384, id_s, steps);
                ptx::mma_commit(&s_full[i]);
                if (i == tiles - 1) ptx::mma_commit(&empty[2 * j % S::kStages]);
            };
            ok = ptx::mbar_wait(q_full, 0, wait_ns) && arrived(0);
            ptx::tc_fence_after();
            for (int i = 0; i < tiles && ok; ++i) scores(i, 0);
            for (int j = 0; j < n && ok; ++j) {
                ok = arrived(2 * j + 1);
                const uint64_t vd = ptx::desc_mn_sw128(stage(2 * j + 1), 16384);
                for (int i = 0; i < tiles && ok; ++i) {
                    ok = ptx::mbar_wait(&p_full[i], j & 1, wait_ns);
                    if (!ok) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int q = 0; q < kKeys / 16; ++q)
                        ptx::mma_f16_ts(tmem + TILES * 128 + i * D, tmem + i * 128 + q * 8, vd + q * 128, id_o, (j | q) != 0);
                    if (i == tiles - 1) ptx::mma_commit(&empty[(2 * j + 1) % S::kStages]);
                    if (j + 1 < n) {
                        if (i == 0) ok = arrived(2 * j + 2);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        scores(i, j + 1);
                    } else {
                        ptx::mma_commit(&o_full[i]);
                    }
                }
            }
            if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
            ptx::mma_commit(drain);
            ptx::mbar_wait(drain, 0, kAttnDrainNs);
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int i = (warp - 2) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        if (i < tiles) {
            const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
            const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + TILES * 128 + i * D;
            const float c = a.scale * kLog2e;
            // P is kept up to 2^8 (kLazy); in fp16 2^7 more, so that small probabilities keep their digits
            constexpr float kUp = std::is_same<T, __half>::value ? 7.f : 0.f;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                ok = __all_sync(FULL_MASK, ptx::mbar_wait(&s_full[i], j & 1, wait_ns));
                if (!ok) break;
                ptx::tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int x = 0; x < 4; ++x) ptx::tmem_ld32(s_at + x * 32, v[x]);
                ptx::tmem_ld_wait();
                const int valid = (int)min((int64_t)kKeys, hi - lo - (int64_t)j * kKeys);
                if (valid < kKeys) {
#pragma unroll
                    for (int x = 0; x < 128; ++x)
                        if (x >= valid) v[x >> 5][x & 31] = 0xff800000u;
                }
                float most[4] = {m, m, m, m};
#pragma unroll
                for (int x = 0; x < 32; ++x) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) most[y] = fmaxf(most[y], __uint_as_float(v[y][x]));
                }
                const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                const bool grow = (top - m) * c > kLazy;  // false where both are -inf
                if (__any_sync(FULL_MASK, grow)) {
                    const float shrink = grow ? ptx::ex2((m - top) * c) : 1.f;
                    if (grow) m = top;
                    l *= shrink;
                    if (j > 0) {
#pragma unroll 1
                        for (int x = 0; x < D; x += 16) {
                            uint32_t o[16];
                            ptx::tmem_ld16(o_at + x, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * shrink);
                            ptx::tmem_st16(o_at + x, o);
                        }
                    }
                }
                const F2 base = both(m == -INFINITY ? 0.f : kUp - m * c), cc = both(c);
                F2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t p[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        F2 e = fma(F2{__uint_as_float(v[x][2 * y]), __uint_as_float(v[x][2 * y + 1])}, cc, base);
                        e = F2{ptx::ex2(e.x), ptx::ex2(e.y)};
                        sum[y & 1] = add(sum[y & 1], e);
                        p[y] = pack2<T>(e.x, e.y);
                    }
                    ptx::tmem_st16(s_at + x * 16, p);
                }
                ptx::tmem_st_wait();
                sum[0] = add(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                if (i == 0 && valid < kKeys) {
                    const int it = 2 * j + 1;
                    ok = __all_sync(FULL_MASK, ptx::mbar_wait(&full[it % S::kStages], (it / S::kStages) & 1, wait_ns));
                    if (!ok) break;
                    attn_clear_rows<S::kBoxes>(ring_base + (uint32_t)(it % S::kStages) * S::kTile, kKeys, valid, r, 128);
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&p_full[i]);
            }
            if (ok && n > 0) ok = __all_sync(FULL_MASK, ptx::mbar_wait(&o_full[i], 0, wait_ns));
            ptx::tc_fence_after();
            if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
            const int pos = r / pk.heads;
            const int64_t row = t.row + i * pk.positions + pos;
            const int head = head0 + r - pos * pk.heads;
            const bool there = ok && pos < pk.positions && row < t.end;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* o = static_cast<T*>(a.o) + row * a.ldo + (int64_t)head * a.d;
            const int64_t at = (blockIdx.z * a.nq + row) * a.hq + head;
            if (there) {
                const float lse = l == 0.f ? -INFINITY : (m * c - kUp + log2f(l)) * kLn2;
                if (a.splits > 1) a.part_lse[at] = lse;
                else a.lse[row * a.hq + head] = lse;
            }
#pragma unroll 1
            for (int x = 0; x < D && ok; x += 32) {
                if (x >= a.d || (n == 0 && a.splits > 1)) break;  // the join passes over a split without keys
                uint32_t v[32];
                if (n > 0) {
                    ptx::tmem_ld32(o_at + x, v);
                    ptx::tmem_ld_wait();
                }
#pragma unroll
                for (int y = 0; y < 32; ++y) v[y] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(v[y]) * inv);
                if (!there) continue;
                if (a.splits > 1) {
#pragma unroll
                    for (int y = 0; y < 32; y += 4)
                        if (x + y < a.d)
                            *reinterpret_cast<uint4*>(a.part + at * a.d + x + y) = make_uint4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                } else {
#pragma unroll
                    for (int y = 0; y < 32; y += 8) {
                        uint4 w;
                        w.x = pack2<T>(__uint_as_float(v[y]), __uint_as_float(v[y + 1]));
                        w.y = pack2<T>(__uint_as_float(v[y + 2]), __uint_as_float(v[y + 3]));
                        w.z = pack2<T>(__uint_as_float(v[y + 4]), __uint_as_float(v[y + 5]));
                        w.w = pack2<T>(__uint_as_float(v[y + 6]), __uint_as_float(v[y + 7]));
                        if (x + y < a.d) *reinterpret_cast<uint4*>(o + x + y) = w;
                    }
                }
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, S::kCols);
    }
}

template <typename T, int D, int TILES>
spc_status launch(const AttnArgs& a, const AttnShape& f, cudaStream_t st)
{
    using S = Shape<D, TILES>;
    CUtensorMap q, k, v;
    if (!attn_tmap<T>(&q, a.q, a.ldq, a.nq, a.hq, a.d, f.heads, f.positions) || !attn_tmap<T>(&k, a.k, a.ldk, a.nk, a.hk, a.d, 1, kKeys) ||
        !attn_tmap<T>(&v, a.v, a.ldv, a.nk, a.hk, a.d, 1, kKeys))
        return SPC_ERR_UNSUPPORTED;
    const int64_t slots = attn_slots(a.nq, a.segments, f.positions * TILES);
    if (slots > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    const spc_status s = allow_smem<k_attn_tc<T, D, TILES>>();
    if (s != SPC_OK) return s;
    return attn_start_kernel<k_attn_tc<T, D, TILES>>(dim3((unsigned)slots, (unsigned)(a.hq / f.heads), a.splits), S::kThreads, S::kSmem,
                                                     st, a, Packing{f.heads, f.positions}, wait_limit_ns(), q, k, v);
}

template <typename T>
spc_status typed(const AttnArgs& a, const AttnShape& f, cudaStream_t st)
{
    if (a.d <= 64) return f.tiles == 2 ? launch<T, 64, 2>(a, f, st) : launch<T, 64, 1>(a, f, st);
    return f.tiles == 2 ? launch<T, 128, 2>(a, f, st) : launch<T, 128, 1>(a, f, st);
}

}  // namespace

spc_status attention_fwd_tc(const AttnArgs& a, spc_dtype dt, cudaStream_t st)
{
    const AttnShape f = attn_shape(a.nq, a.segments, a.hq, a.hk);
    return dt == SPC_F16 ? typed<__half>(a, f, st) : typed<__nv_bfloat16>(a, f, st);
}

}  // namespace spc
