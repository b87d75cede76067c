// attention_tc.cu -- the forward pass of attention over segments on the 5th-generation tensor cores.
//
// A block keeps TILES tiles of 128 query rows (the positions of a segment, and the query heads that share a key head
// beside one another, so that keys are read once for all of them) and walks over the segment's keys 64 at a time:
//   four warps for each tile take S, a thread to a row: running maximum, exponentials, P as 16 bits in the place of S;
//   a warp loads the queries once and keys and values into a ring of stages (TMA);
//   two warps for each tile issue S = Q K^T into tensor memory, and O += P V with P from tensor memory.  A warp's waits
//     queue up behind its own products: with one warp for all of them the tensor cores idled half of the time
//     (32,768 rows in 2 samples, 8 heads of 128: 2,005 us against 1,371).
// S has two buffers a tile, so the next scores are there when a tile's exponentials are done, and with two tiles (or two
// blocks on an SM) the products of one run while the other's exponentials are taken.  O stays in tensor memory; it is
// rescaled only when a row's maximum has grown by more than 2^8, so almost never after the first tiles
// (sums and P carry the same factor, which the end divides out).
//
// Heads of 128: 1,620 to 1,660 TFLOP/s over 16,384 rows a sample, 85% of measured cuBLAS, bound by the tensor cores at the
// pace of 64-column products (a product of 128 x 64 x 16 takes what its 6 KB take to leave shared memory, 48 cycles for 32
// of arithmetic).  Heads of 64: 890 to 980, bound by the way from scores through exponentials and sums back to free scores, of which
// two blocks an SM hide a part: exponentials fill 40% of their unit's time, instructions 53%, products 39%.  Tried and slower for heads
// of 64: no running maximum but a check of each step's sum (613 us against 634, but 1,468 against 1,385 for heads
// of 128), eight warps a tile (616 against 640), three score buffers (667), 128 keys a step (887).
//
// Every wait is bounded by the library's wait limit; one that runs out sets SPC_ERR_TIMEOUT, and each role then
// waits (bounded) for what it has in flight itself before the block frees its tensor memory and returns.
#include "attention_tc.cuh"

namespace spc {

namespace {

constexpr int kKeys = 64;        // keys of a step
constexpr float kLazy = 8.f;     // a maximum may grow by this much (log2) before sums are rescaled

template <int D, int TILES>
struct Shape {
    static constexpr int kBoxes = D / 64;
    static constexpr int kTile = 128 * 128 * kBoxes;          // bytes of a tile's queries
    static constexpr int kPart = kKeys * 128 * kBoxes;        // bytes of a step's keys, or values
    static constexpr int kStage = 2 * kPart;                  // the values of a step, the keys of the next but one
    static constexpr int kStages = TILES == 1 && D == 128 ? 2 : 4;  // what fits beside a second block
    static constexpr int kLoad = 4 * TILES;                   // the warp that loads; after it those that issue
    static constexpr int kThreads = 32 * (kLoad + 1 + 2 * TILES);
    static constexpr int kCols = TILES == 2 ? 512 : 256;      // tensor memory: 128 of scores and D of sums a tile
    static constexpr int kBars = 3 * kStages + 1 + 8 * TILES;
    static constexpr size_t kSmem = 1024 + (size_t)TILES * kTile + (size_t)kStages * kStage + 8 * kBars + 16;
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
    // a stage: the values of a step, then the keys of the next but one (the last two begin with those of steps 0 and 1)
    uint8_t* ring = smem + TILES * S::kTile;
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)S::kStages * S::kStage);
    uint64_t* k_empty = full + S::kStages;
    uint64_t* v_empty = k_empty + S::kStages;
    uint64_t* q_full = v_empty + S::kStages;
    uint64_t* drain = q_full + 1;             // [tile][2]
    uint64_t* s_full = drain + 2 * TILES;     // [tile][buffer]: the scores of a step
    uint64_t* p_full = s_full + 2 * TILES;    // [tile][buffer]: its probabilities
    uint64_t* o_full = p_full + 2 * TILES;    // [tile][buffer]: the sums with them
    uint32_t* s_ctrl = reinterpret_cast<uint32_t*>(o_full + 2 * TILES);
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
            ptx::mbar_init(&k_empty[s], tiles);
            ptx::mbar_init(&v_empty[s], tiles);
        }
        ptx::mbar_init(q_full, 1);
        for (int i = 0; i < 2 * TILES; ++i) {
            ptx::mbar_init(&drain[i], 1);
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_full[i], 4);
            ptx::mbar_init(&o_full[i], 1);
        }
        ptx::mbar_init_fence();
    }
    if (warp == S::kLoad) {
        ptx::tmem_alloc(s_ctrl, S::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_ctrl[0];
    const uint32_t q_base = ptx::smem_u32(smem), ring_base = ptx::smem_u32(ring);
    bool ok = true;


    if (warp == S::kLoad) {
        // ------------------------------------------------------------ loads
        if (n > 0) {
            auto load = [&](uint32_t to, const CUtensorMap* map, int step, uint64_t* bar) {
#pragma unroll
                for (int b = 0; b < S::kBoxes; ++b)
                    ptx::tma_load3d<1>(to + b * (kKeys * 128), map, b * 64, kv, (int32_t)lo + step * kKeys, ptx::smem_u32(bar));
            };
            if (attn_elect()) {
                ptx::mbar_arrive_expect_tx(q_full, (uint32_t)pk.heads * pk.positions * 128 * S::kBoxes * tiles + S::kPart * min(n, 2));
                for (int i = 0; i < tiles; ++i)
                    for (int b = 0; b < S::kBoxes; ++b)
                        ptx::tma_load3d<1>(q_base + i * S::kTile + b * 16384, &map_q, b * 64, head0, (int32_t)(t.row + i * pk.positions),
                                           ptx::smem_u32(q_full));
                for (int j = 0; j < min(n, 2); ++j) load(ring_base + (S::kStages - 2 + j) * S::kStage + S::kPart, &map_k, j, q_full);
            }
            __syncwarp();
            int j = 0;
            for (; j < n; ++j) {
                // freed once for each step that used it, and the keys' part of the last two by steps 0 and 1 besides
                const int s = j % S::kStages, round = j / S::kStages, keys = round + (s >= S::kStages - 2);
                if (round > 0) ok = attn_wait(&v_empty[s], (round - 1) & 1, wait_ns);
                if (keys > 0 && ok) ok = attn_wait(&k_empty[s], (keys - 1) & 1, wait_ns);
                if (!ok) break;
                if (attn_elect()) {
                    const uint32_t to = ring_base + s * S::kStage;
                    ptx::mbar_arrive_expect_tx(&full[s], j + 2 < n ? S::kStage : S::kPart);
                    load(to, &map_v, j, &full[s]);
                    if (j + 2 < n) load(to + S::kPart, &map_k, j + 2, &full[s]);
                }
                __syncwarp();
            }
            if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
            // what is in flight has to land before the block's shared memory goes
            ptx::mbar_wait(q_full, 0, kAttnDrainNs);
            for (int i = max(j - S::kStages, 0); i < j; ++i) ptx::mbar_wait(&full[i % S::kStages], (i / S::kStages) & 1, kAttnDrainNs);
        }
    } else if (warp > S::kLoad) {
        // ------------------------------------------------------------- MMAs
        const int i = (warp - S::kLoad - 1) >> 1;
        const bool scores = (warp - S::kLoad) & 1;
        if (n > 0 && i < tiles) {
            const int steps = (a.d + 15) / 16;
            const uint32_t s_at = tmem + i * 128, o_at = tmem + TILES * 128 + i * D;
            if (scores) {
                const uint32_t idesc = ptx::idesc_make(AttnFmt<T>::v, 128, kKeys);
                const uint64_t q_desc = ptx::desc_k_sw128(q_base + i * S::kTile), k_desc = ptx::desc_k_sw128(ring_base + S::kPart);
                ok = attn_wait(q_full, 0, wait_ns);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = (j + S::kStages - 2) % S::kStages;
                    // in the place of P, once the sums of step j - 2 have it
                    if (j >= 2)
                        ok = attn_wait(&full[s], ((j - 2) / S::kStages) & 1, wait_ns) && attn_wait(&o_full[2 * i + (j & 1)], ((j - 2) >> 1) & 1, wait_ns);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (attn_elect()) {
                        attn_mma_ss<D / 16>(s_at + (j & 1) * 64, q_desc, 16384, k_desc + s * (S::kStage >> 4), kKeys * 128, idesc, steps);
                        ptx::mma_commit(&s_full[2 * i + (j & 1)]);
                        ptx::mma_commit(&k_empty[s]);
                    }
                    __syncwarp();
                }
            } else {
                const uint32_t idesc = ptx::idesc_make(AttnFmt<T>::v, 128, steps * 16) | 1u << 16;
                const uint64_t v_desc = ptx::desc_mn_sw128(ring_base, kKeys * 128);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = j % S::kStages;
                    ok = attn_wait(&full[s], (j / S::kStages) & 1, wait_ns) && attn_wait(&p_full[2 * i + (j & 1)], (j >> 1) & 1, wait_ns);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (attn_elect()) {
#pragma unroll
                        for (int q = 0; q < kKeys / 16; ++q)
                            ptx::mma_f16_ts(o_at, s_at + (j & 1) * 64 + q * 8, v_desc + s * (S::kStage >> 4) + q * 128, idesc, q > 0 || j > 0);
                        ptx::mma_commit(&o_full[2 * i + (j & 1)]);
                        ptx::mma_commit(&v_empty[s]);
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
            uint64_t* mine = &drain[2 * i + scores];
            if (attn_elect()) ptx::mma_commit(mine);
            __syncwarp();
            ptx::mbar_wait(mine, 0, kAttnDrainNs);
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int i = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        if (i < tiles) {
            const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
            const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + TILES * 128 + i * D;
            const float c = a.scale * kLog2e;
            // P is kept up to 2^8 (kLazy); in fp16 2^7 more, so that small probabilities keep their digits
            constexpr float kUp = std::is_same<T, __half>::value ? 7.f : 0.f;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                ok = attn_wait(&s_full[2 * i + (j & 1)], (j >> 1) & 1, wait_ns);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t at = s_at + (j & 1) * 64;
                uint32_t v[2][32];
                ptx::tmem_ld32(at, v[0]);
                ptx::tmem_ld32(at + 32, v[1]);
                ptx::tmem_ld_wait();
                const int valid = (int)min((int64_t)kKeys, hi - lo - (int64_t)j * kKeys);
                if (valid < kKeys) {
#pragma unroll
                    for (int x = 0; x < kKeys; ++x)
                        if (x >= valid) v[x >> 5][x & 31] = 0xff800000u;
                }
                float most[4] = {m, m, m, m};
#pragma unroll
                for (int x = 0; x < 8; ++x) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        most[y] = ptx::max3(most[y], __uint_as_float(v[y >> 1][4 * x + 2 * (y & 1)]), __uint_as_float(v[y >> 1][4 * x + 2 * (y & 1) + 1]));
                }
                const float top = fmaxf(ptx::max3(most[0], most[1], most[2]), most[3]);
                const bool grow = (top - m) * c > kLazy;  // false where both are -inf
                if (__any_sync(FULL_MASK, grow)) {
                    const float shrink = grow ? ptx::ex2((m - top) * c) : 1.f;
                    if (grow) m = top;
                    l *= shrink;
                    if (j > 0) {
                        // the sums of step j - 1 (the scores of step j - 1 showed those of step j - 3, so the parity is not mistaken)
                        ok = attn_wait(&o_full[2 * i + ((j - 1) & 1)], ((j - 1) >> 1) & 1, wait_ns);
                        if (!ok) break;
                        ptx::tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < D; x += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld32(o_at + x, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * shrink);
                            ptx::tmem_st32(o_at + x, o);
                        }
                    }
                }
                const F2 base = both(m == -INFINITY ? 0.f : kUp - m * c), cc = both(c);
                F2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
                uint32_t p[32];
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                    F2 e = fma(F2{__uint_as_float(v[y >> 4][2 * (y & 15)]), __uint_as_float(v[y >> 4][2 * (y & 15) + 1])}, cc, base);
                    e = F2{ptx::ex2(e.x), ptx::ex2(e.y)};
                    sum[y & 1] = add(sum[y & 1], e);
                    p[y] = pack2<T>(e.x, e.y);
                }
                ptx::tmem_st32(at, p);
                sum[0] = add(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                ptx::tmem_st_wait();
                if (valid < kKeys) {  // by each tile's warps: its own products wait for them alone
                    ok = attn_wait(&full[j % S::kStages], (j / S::kStages) & 1, wait_ns);
                    if (!ok) break;
                    attn_clear_rows<S::kBoxes>(ring_base + (uint32_t)(j % S::kStages) * S::kStage, kKeys, valid, r, 128);
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&p_full[2 * i + (j & 1)]);
            }
            if (ok && n > 0) ok = attn_wait(&o_full[2 * i + ((n - 1) & 1)], ((n - 1) >> 1) & 1, wait_ns);
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
                __syncwarp();
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
    if (warp == S::kLoad) {
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
    if (a.d <= 64) return launch<T, 64, 1>(a, f, st);
    return f.tiles == 2 ? launch<T, 128, 2>(a, f, st) : launch<T, 128, 1>(a, f, st);
}

}  // namespace

spc_status attention_fwd_tc(const AttnArgs& a, spc_dtype dt, cudaStream_t st)
{
    const AttnShape f = attn_shape(a.nq, a.segments, a.hq, a.hk, a.d);
    return dt == SPC_F16 ? typed<__half>(a, f, st) : typed<__nv_bfloat16>(a, f, st);
}

}  // namespace spc
