// Chunk attention, bf16: the products on tcgen05 with logits, probabilities and outputs
// in tensor memory. chunk_attn.cuh states the mathematics and the split over the GPU; a
// step here is 128 tokens, a unit two MMA tiles of 128 rows (kTwo), or one where every
// chunk of the call fits into it (max_new * G <= 128, decode included).
//
// Warps. 0-3 and 4-7: softmax of two streams (one row per thread); 8: TMA (K and V tiles
// page by page into a ring, query tiles; no multicast); 9: issues the MMAs, and looks over
// the V tiles that some row does not see whole.
//   S = Q K^T       M128 N128 Kd, both operands in shared memory as TMA wrote them
//   P = exp2(sl2 S - m), rounded to bf16 over S's columns in tensor memory
//   O += P V        M128 Nd K128, P from tensor memory, V as TMA wrote it (N-major)
// The streams alternate on the tensor pipe: one's products run while the other's softmax
// does. In a unit of two query tiles a stream is a tile; in a unit of one, it is every other
// step of that tile, with an O of its own, and stream 0's epilogue adds the two (both stand
// in the same lanes). A step's softmax takes longer than its K and V take to come from
// memory: one stream alone bounds a decode by its exponentials (16 a clock and SM).
// The maximum a row's sums are scaled by follows the running maximum only when that has
// grown by more than 2^8: until then the sums are merely larger, not less exact, and
// the rescale of O (a pass over tensor memory) is skipped. l sums the probabilities
// before they are rounded; the products see them rounded to bf16 (half a step, 2^-8
// relative, averaged over the tokens), which is what the MMA's operand type allows
// without a second product.
//
// Tokens past the sequence's end may be anything, NaN included, and so may tokens that
// come after a row's own: logits there are replaced by -inf. Their V rows meet a
// probability of zero, but 0 * inf is NaN: rows past the end are zeroed in the tile, and
// in tiles on the diagonal infinities and NaN are taken out of V and noted per dimension
// (the first token that holds one, by kind), and the epilogue adds them to the rows that
// see that token.
#include <algorithm>
#include <atomic>

#include "chunk_attn.cuh"

namespace spla {

constexpr int kTcThreads = 384;
constexpr int kTcSmem = 227 * 1024;
// Registers: the kernel is launched with 168 a thread; the softmax warps (a row of logits
// each thread) take 216 and the other four give theirs down to 72. The shares add up to
// the launch's: 256 * 216 + 128 * 72 = 384 * 168.
// The two sides share no code after the split, their ends included: code common to both
// is compiled for the larger side's registers, and a warp of the smaller side that runs
// it overwrites registers that are a softmax warp's by then.
constexpr int kTcRegs = 168, kTcRegsMore = 216, kTcRegsLess = 72;
static_assert(256 * kTcRegsMore + 128 * kTcRegsLess <= kTcThreads * kTcRegs, "register shares");
constexpr float kTcLazy = 8.f;               // log2 growth of a maximum that is let stand

template <int D, bool kTwo>
struct TcShape {
    static constexpr int kQTiles = kTwo ? 2 : 1;
    static constexpr int kHalves = D / 64;                   // 64-dimension boxes across a row
    static constexpr int kTileBytes = kTcTile * D * 2;       // a K, V or Q tile
    static constexpr int kBox = 8192;                        // 64 tokens x 64 dims
    static constexpr int kCtl = 3008;                        // barriers and notes
    // Query tiles of two units where they fit beside the ring: short units then follow one
    // another without a wait for their queries.
    static constexpr int kQBufs = D == 64 ? 2 : 1;
    static constexpr int kFit = (kTcSmem - kCtl) / kTileBytes - kQTiles * kQBufs;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr int kRows = 128 * kQTiles;
    static constexpr size_t kSmem = kCtl + (size_t)(kQTiles * kQBufs + kStages) * kTileBytes;
    static_assert(kStages >= 4, "the ring holds two steps");
    static_assert(kSmem <= kTcSmem, "shared memory");
};

// ------------------------------------------------------------------ tcgen05 plumbing
__device__ __forceinline__ void tcf_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcf_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle, 1024-byte aligned 8-row atoms
// (version 1). K-major: rows of 64 elements, 8-row groups 1024 bytes apart. MN-major:
// 64-element atoms `lbo` bytes apart, 8-row groups of K 1024 bytes apart.
// The words: address and lbo in units of 16 bytes; the rest is constant.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t tc_desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | (lbo >> 4) << 16;
}
__device__ __forceinline__ uint64_t tc_desc(uint32_t lo) {
    return (uint64_t)kDescHi << 32 | lo;
}

// One thread of the converged warp; the others skip what it guards.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// kind::f16, fp32 accumulator, bf16 operands, A K-major, M = 128.
constexpr uint32_t tc_idesc(int n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_u32(bar)) : "memory");
}

// N consecutive columns of this thread's TMEM lane, waited for: the load is asynchronous,
// so the wait stands in the same statement and nothing can use the registers before it.
__device__ __forceinline__ void tm_ld32(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
          "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
          "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
          "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
          "=f"(v[30]), "=f"(v[31])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tm_ld128(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
          "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
          "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
          "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
          "=f"(v[30]), "=f"(v[31]), "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]),
          "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]), "=f"(v[41]),
          "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
          "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]),
          "=f"(v[54]), "=f"(v[55]), "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]),
          "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]), "=f"(v[64]), "=f"(v[65]),
          "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
          "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]),
          "=f"(v[78]), "=f"(v[79]), "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]),
          "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]), "=f"(v[88]), "=f"(v[89]),
          "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]),
          "=f"(v[96]), "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]),
          "=f"(v[102]), "=f"(v[103]), "=f"(v[104]), "=f"(v[105]), "=f"(v[106]), "=f"(v[107]),
          "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]), "=f"(v[112]), "=f"(v[113]),
          "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]), "=f"(v[119]),
          "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]),
          "=f"(v[126]), "=f"(v[127])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
           "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
           "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
           "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
           "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
           "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
           "r"(r[14]), "r"(r[15]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tm_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_q(void* dst, const void* tmap, uint64_t* bar, int32_t x,
                                      int32_t head, int32_t tok, int32_t seq) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        :: "r"(smem_u32(dst)), "l"(tmap), "r"(smem_u32(bar)), "r"(x), "r"(head), "r"(tok), "r"(seq)
        : "memory");
}

template <int D, bool kTwo> using TcWalk = Walk<kTcTile, TcCost<D>, !kTwo>;

template <int D, bool kTwo>
struct TcNotes {                              // control block in shared memory
    uint64_t kv_full[8], kv_empty[8];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2], o_done[2]; // by stream
    uint64_t m_full, m_empty, fin;            // stream 1's sums for stream 0's epilogue
    int64_t scan[kTcThreads / 32];
    TcWalk<D, kTwo> start;
    int64_t run;                              // C
    uint32_t tmem;
    int32_t nf_seg;                           // segment whose infinities and NaN are noted
    int32_t epi[2];                           // by stream: warps past an epilogue, over all segments
    int32_t first[3][128];                    // first token with +inf, -inf, NaN, per dimension
    float m1[128], l1[128];
};
static_assert(sizeof(TcNotes<128, true>) <= 3008, "control block");

// Bounded waits. A role may sit out another's whole run (thousands of steps), so the
// bound is far: seconds at the shortest poll. (Inlined at every use: kept small.)
constexpr uint32_t kTcPolls = 1u << 27;
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
#pragma unroll 1
    for (uint32_t i = 0; i < kTcPolls; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    set_status(status, SPLA_DEV_TIMEOUT);
    return false;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int D, bool kTwo>
__global__ void __launch_bounds__(kTcThreads, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const CacheView c, const ChunkArgs a) {
    using S = TcShape<D, kTwo>;
    extern __shared__ __align__(1024) unsigned char tc_smem[];      // swizzle atoms are 1024 bytes
    unsigned char* qtile = tc_smem;
    unsigned char* ring = tc_smem + S::kQTiles * S::kQBufs * S::kTileBytes;
    TcNotes<D, kTwo>* nt = reinterpret_cast<TcNotes<D, kTwo>*>(ring + S::kStages * S::kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = c.group, lgG = G >> 1;               // 1, 2 or 4
    const int per_tile = 128 >> lgG;                      // query tokens of a tile
    const int U = per_tile * S::kQTiles;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&nt->kv_full[s], 1);
            mbar_init(&nt->kv_empty[s], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&nt->q_full[w], 1);
            mbar_init(&nt->q_empty[w], 1);
        }
        mbar_init(&nt->m_full, 4);
        mbar_init(&nt->m_empty, 4);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&nt->s_full[w], 1);
            mbar_init(&nt->p_full[w], 4);
            mbar_init(&nt->o_done[w], 1);
        }
        mbar_init(&nt->fin, 1);
        fence_barrier_init();
        prefetch_tmap(&tq);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
        nt->nf_seg = -1;
        nt->epi[0] = nt->epi[1] = 0;
        nt->start.j = 0;
        nt->start.F = nt->start.end = 0;
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_u32(&nt->tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();

    tcf_before();
    find_run<kTcThreads>(c, a, per_tile, U, nt->scan, nt->first[0], &nt->start, &nt->run);
    tcf_after();
    const uint32_t tmem = nt->tmem;
    TcWalk<D, kTwo> wk = nt->start;

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kTcRegsLess));
    if (warp == 8) {
        // ---------------------------------------------------------- TMA producer
        int it = 0, seg = 0;                            // ring slots filled, segments
        bool ok = true;
        const int32_t none = (int32_t)((int64_t)c.num_phys * c.hkv * c.bs);   // reads as zeros
        const int two = c.bs >> 7;                      // whether a page has two 64-token rows
#pragma unroll 1
        while (ok && wk.next(c, a, per_tile, U)) {
            const int32_t* row = c.table + (int64_t)wk.b * c.mbp;
            const int nu = (wk.L + 63) / 64;            // 64-token rows the sequence holds
            int32_t ys = none;
#pragma unroll 1
            for (int j = wk.j0; j < wk.j1; ++j) {
                const int k = (j - wk.j0) & 15;
                if (k == 0) {                           // 16 steps' page rows at a time
                    const int u = 2 * j + lane;
                    ys = none;
                    if (u < nu) {
                        const int32_t phys = row[u >> two];
                        if (phys >= 0 && phys < c.num_phys)
                            ys = (phys * c.hkv + wk.h) * c.bs + (u & two) * 64;
                        else
                            set_status(a.status, SPLA_DEV_BAD_BLOCK_TABLE);
                    }
                }
                const int32_t y0 = __shfl_sync(0xffffffffu, ys, 2 * k);
                const int32_t y1 = __shfl_sync(0xffffffffu, ys, 2 * k + 1);
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const int s = it % S::kStages;
                    if (it >= S::kStages)
                        ok = tc_wait(&nt->kv_empty[s], (it / S::kStages - 1) & 1, a.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        unsigned char* st = ring + s * S::kTileBytes;
                        mbar_arrive_expect_tx(&nt->kv_full[s], S::kTileBytes);
                        for (int x = 0; x < S::kHalves; ++x) {
                            tma_load_2d(st + x * 16384, kv ? &tv : &tk, &nt->kv_full[s], 64 * x, y0);
                            tma_load_2d(st + x * 16384 + 8192, kv ? &tv : &tk, &nt->kv_full[s],
                                        64 * x, y1);
                        }
                    }
                    // the unit's queries: behind its first K where their buffer is free from the
                    // start, else behind its first V, which need not wait for the unit before to
                    // be done with its own
                    if (j != wk.j0 || kv != (seg >= S::kQBufs)) continue;
                    const int qs = seg % S::kQBufs;
                    if (seg >= S::kQBufs)
                        ok = tc_wait(&nt->q_empty[qs], (seg / S::kQBufs - 1) & 1, a.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        const int tiles = wk.pair(per_tile, U) ? S::kQTiles : 1;
                        mbar_arrive_expect_tx(&nt->q_full[qs], tiles * S::kTileBytes);
#pragma unroll 1
                        for (int w = 0; w < tiles; ++w)
                            for (int x = 0; x < S::kHalves; ++x)
                                tma_q(qtile + (qs * S::kQTiles + w) * S::kTileBytes + x * 16384, &tq,
                                      &nt->q_full[qs], 64 * x, wk.h * G, wk.qb * U + w * per_tile,
                                      wk.b);
                    }
                }
                if (!ok) break;
            }
            ++seg;
        }
        // the copies in flight have landed before the CTA may leave
#pragma unroll 1
        for (int i = max(0, it - S::kStages); i < it; ++i)
            mbar_wait_bounded(&nt->kv_full[i % S::kStages], (i / S::kStages) & 1);
#pragma unroll 1
        for (int i = max(0, seg - S::kQBufs); i < seg; ++i)
            mbar_wait_bounded(&nt->q_full[i % S::kQBufs], (i / S::kQBufs) & 1);
    } else if (warp == 9) {
        // ---------------------------------------------------------- MMA issuer
        constexpr uint32_t kIdS = tc_idesc(128, false), kIdO = tc_idesc(D, true);
        const uint32_t q0 = smem_u32(qtile), r0 = smem_u32(ring);
        int it = 0, seg = 0;
        uint32_t ps = 0;                                // parities of the probabilities awaited
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool r = __all_sync(0xffffffffu, tc_wait(bar, parity, a.status));
            tcf_after();
            return r;
        };
        auto full = [&](int i) { return wait(&nt->kv_full[i % S::kStages], (i / S::kStages) & 1); };
        // Descriptor words and addresses are made by the whole warp from lane 0's values, so
        // that they stand in uniform registers where the MMAs want them: made within the
        // elected thread's branch, each MMA took twice as long to issue as to run.
        auto uni = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
        auto commit = [&](uint64_t* bar) {
            if (elect_one()) tc_commit(bar);
        };
        // S of the query tile at qs by ring slot i, for stream w
        auto do_s = [&](int qs, int w, int i) {
            const uint32_t kd = uni(tc_desc_lo(r0 + (i % S::kStages) * S::kTileBytes, 16));
            const uint32_t qd = uni(tc_desc_lo(q0 + qs * S::kTileBytes, 16));
            const uint32_t dst = uni(tmem + 128 * w);
            uint64_t* done = &nt->s_full[w];
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss(dst, tc_desc(qd + off), tc_desc(kd + off), kIdS, kk != 0);
                }
                tc_commit(done);
            }
        };
        auto do_o = [&](int w, int i, bool first) {
            const uint32_t vd = uni(tc_desc_lo(r0 + (i % S::kStages) * S::kTileBytes, 16384));
            const uint32_t dst = uni(tmem + 256 + 128 * w), src = uni(tmem + 128 * w);
            const uint32_t acc = uni(first ? 0u : 1u);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTcTile / 16; ++kk)
                    mma_ts(dst, src + 8 * kk, tc_desc(vd + kk * (2048 >> 4)), kIdO,
                           kk != 0 ? 1u : acc);
            }
        };
        auto p_wait = [&](int w) {                      // ps: a phase bit per stream
            const bool r = wait(&nt->p_full[w], (ps >> w) & 1);
            ps ^= 1u << w;
            return r;
        };
        // V of step j is in; where some row does not see all of it, its rows past the
        // sequence are zeroed and its infinities and NaN noted and taken out. The softmax of
        // the step runs meanwhile.
        auto v_wait = [&](int j, int i) {
            if (!full(i)) return false;
            if ((int64_t)(j + 1) * kTcTile <= wk.L - wk.n + (int64_t)wk.qb * U + 1) return true;
            unsigned char* st = ring + (i % S::kStages) * S::kTileBytes;
            const int held = (int)min((int64_t)kTcTile, wk.L - (int64_t)j * kTcTile);
            if (held < kTcTile) {                       // rows past the sequence
                const int n16 = (kTcTile - held) * 8;
#pragma unroll 1
                for (int x = lane; x < n16 * S::kHalves; x += 32)
                    *(reinterpret_cast<uint4*>(st + (x / n16) * 16384) + held * 8 + x % n16) =
                        make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            }
            uint32_t any = 0;                           // an exponent of all ones carries out
            const uint4* p = reinterpret_cast<const uint4*>(st) + lane;
#pragma unroll 1
            for (int x = 0; x < kTcTile * S::kHalves * 8 / 32; x += 8) {
                uint4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = p[(x + u) * 32];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    any |= ((v[u].x & 0x7f807f80u) + 0x00800080u) | ((v[u].y & 0x7f807f80u) + 0x00800080u) |
                           ((v[u].z & 0x7f807f80u) + 0x00800080u) | ((v[u].w & 0x7f807f80u) + 0x00800080u);
            }
            if (__any_sync(0xffffffffu, any & 0x80008000u)) {
                if (nt->nf_seg != seg) {
                    // the rows of the segments before have read their notes, those of either
                    // stream: in segments of one step stream 1 runs ahead
                    const volatile int32_t* epi = nt->epi;
                    uint32_t polls = 0;
#pragma unroll 1
                    while ((epi[0] < 4 * seg || epi[1] < 4 * seg) && ++polls < kTcPolls) {}
                    if (polls == kTcPolls) set_status(a.status, SPLA_DEV_TIMEOUT);
                    __syncwarp();
#pragma unroll 1
                    for (int x = lane; x < 3 * 128; x += 32) nt->first[x / 128][x % 128] = 0x7fffffff;
                    // the flag behind the reset: stream 0 may be in its epilogue already where
                    // only stream 1 needs this tile
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0) *(volatile int32_t*)&nt->nf_seg = seg;
                    __syncwarp();
                }
                // 16-byte chunk ch of row r sits at position ch ^ (r % 8) of its 128-byte row
#pragma unroll 1
                for (int x = lane; x < kTcTile * S::kHalves * 8; x += 32) {
                    const int r = (x >> 3) & 127, dim0 = (x >> 10) * 64 + (((x & 7) ^ (r & 7)) << 3);
                    uint32_t* p = reinterpret_cast<uint32_t*>(st + x * 16);
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t h16 = (p[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                        if ((h16 & 0x7f80u) != 0x7f80u) continue;
                        const int kind = (h16 & 0x7fu) ? 2 : (h16 >> 15);
                        atomicMin(&nt->first[kind][dim0 + e], j * kTcTile + r);
                        p[e >> 1] &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
                    }
                }
            }
            fence_proxy_async();
            __syncwarp();
            return true;
        };
#pragma unroll 1
        while (ok && wk.next(c, a, per_tile, U)) {
            const int qi = seg % S::kQBufs, qt = qi * S::kQTiles;
            uint64_t* q_empty = &nt->q_empty[qi];
            if (!(ok = wait(&nt->q_full[qi], (seg / S::kQBufs) & 1))) break;
            const int nj = wk.j1 - wk.j0;
            // slot it + 2 i is K of step i, it + 2 i + 1 its V
            if (kTwo && wk.pair(per_tile, U)) {
                const int e[2] = {wk.tile_end(0, per_tile, U), wk.tile_end(1, per_tile, U)};
                if (!(ok = full(it))) break;
#pragma unroll 1
                for (int w = 0; w < 2; ++w)
                    if (wk.j0 < (w ? e[1] : e[0])) do_s(qt + w, w, it);
                commit(&nt->kv_empty[it % S::kStages]);
                if (nj == 1) commit(q_empty);
#pragma unroll 1
                for (int i = 0; i < nj && ok; ++i) {
                    const int j = wk.j0 + i, iv = it + 2 * i + 1, ik = iv + 1;
                    if (!(ok = v_wait(j, iv))) break;
                    if (i + 1 < nj && !(ok = full(ik))) break;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int ew = w ? e[1] : e[0];
                        if (j >= ew) continue;
                        if (!(ok = p_wait(w))) break;
                        do_o(w, iv, i == 0);
                        if (j + 1 < ew) do_s(qt + w, w, ik);
                        else commit(&nt->o_done[w]);
                    }
                    commit(&nt->kv_empty[iv % S::kStages]);
                    if (i + 1 < nj) commit(&nt->kv_empty[ik % S::kStages]);
                    if (i + 2 == nj) commit(q_empty);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < 2 && i < nj && ok; ++i) {
                    if (!(ok = full(it + 2 * i))) break;
                    do_s(qt, i, it + 2 * i);
                    commit(&nt->kv_empty[(it + 2 * i) % S::kStages]);
                    if (i + 1 == nj) commit(q_empty);
                }
#pragma unroll 1
                for (int i = 0; i < nj && ok; ++i) {
                    const int w = i & 1, iv = it + 2 * i + 1, ik = iv + 3;
                    if (!(ok = v_wait(wk.j0 + i, iv))) break;
                    if (!(ok = p_wait(w))) break;
                    do_o(w, iv, i < 2);
                    if (i + 2 >= nj) commit(&nt->o_done[w]);
                    commit(&nt->kv_empty[iv % S::kStages]);
                    if (i + 2 < nj) {
                        if (!(ok = full(ik))) break;
                        do_s(qt, w, ik);
                        commit(&nt->kv_empty[ik % S::kStages]);
                        if (i + 3 == nj) commit(q_empty);
                    }
                }
            }
            it += 2 * nj;
            ++seg;
        }
        // no MMA of this CTA is in flight once the last commit has fired
        commit(&nt->fin);
        tc_wait(&nt->fin, 0, a.status);
    }
    tcf_before();
    asm volatile("bar.sync 1, %0;" :: "n"(kTcThreads) : "memory");
    if (warp == 9) {
        tcf_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;"
                     :: "r"(tmem) : "memory");
    }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kTcRegsMore));
    {
        // ---------------------------------------------------------- softmax and epilogue
        const int w = warp >> 2;                        // stream
        const int r = tid & 127;                        // row of the tile = TMEM lane
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;       // lane quarter, in the address
        const uint32_t tO = tmem + 256 + 128 * w + lanes;
        int sc = 0, oc = 0, mc = 0;                     // steps, segments with steps, joins
        int seg = 0;
        bool ok = true;
        ChunkCut cut = {};
#pragma unroll 1
        while (ok && wk.next(c, a, per_tile, U)) {
            // a pair: stream w is query tile w, every step; one tile: every other step of it
            const bool pair = kTwo && wk.pair(per_tile, U);
            const int t0 = wk.qb * U + (pair ? w * per_tile : 0);
            const int tok = t0 + (r >> lgG);                 // query token of this row
            const bool live = tok < wk.n;
            const int pos = wk.L - wk.n + tok;
            const int lo_pos = wk.L - wk.n + t0;        // of the tile's first row
            const bool warp_live = t0 + (((warp & 3) * 32) >> lgG) < wk.n;
            const int first_j = wk.j0 + (pair ? 0 : w), by = pair ? 1 : 2;
            const int e = pair ? wk.tile_end(w, per_tile, U) : wk.j1;
            float m = -SPLA_INF, l = 0.f;
#pragma unroll 1
            for (int j = first_j; j < e; j += by, ++sc) {
                ok = tc_wait(&nt->s_full[w], sc & 1, a.status);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (warp_live) {
                    tcf_after();
                    const uint32_t tS = tmem + 128 * w + lanes;
                    float s[128];
                    tm_ld128(tS, s);
                    if ((int64_t)(j + 1) * kTcTile > lo_pos + 1) {
                        const int lim = pos - j * kTcTile;
#pragma unroll
                        for (int i = 0; i < 128; ++i) s[i] = i <= lim ? s[i] : -SPLA_INF;
                    }
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int i = 4; i < 128; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mx[k] = i + 4 + k < 128 ? max3(mx[k], s[i + k], s[i + 4 + k])
                                                    : fmaxf(mx[k], s[i + k]);
                    const float top = fmaxf(max3(mx[0], mx[1], mx[2]), fmaxf(mx[3], m));
                    // the scale of the sums moves where there are none yet, or the maximum
                    // has outgrown it
                    const bool fresh = m == -SPLA_INF;
                    const bool grow = !fresh && (top - m) * a.sl2 > kTcLazy;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? ex2((m - top) * a.sl2) : 1.f;
                        l *= f;
                        // (the product of this stream's last step is done: S came after it)
#pragma unroll 1
                        for (int i = 0; i < D; i += 32) {
                            float o[32];
                            tm_ld32(tO + i, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= f;
                            tm_st32(tO + i, reinterpret_cast<uint32_t*>(o));
                        }
                    }
                    if (fresh || grow) m = top;
                    const float m2 = m == -SPLA_INF ? 0.f : m * a.sl2;
                    const float2 sl = make_float2(a.sl2, a.sl2), mm = make_float2(-m2, -m2);
                    float2 sum = make_float2(0.f, 0.f), sum1 = sum;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float2 p = fma2(make_float2(s[32 * k + i], s[32 * k + i + 1]), sl, mm);
                            float2 q = fma2(make_float2(s[32 * k + i + 2], s[32 * k + i + 3]), sl, mm);
                            p = make_float2(ex2(p.x), ex2(p.y));
                            q = make_float2(ex2(q.x), ex2(q.y));
                            sum = add2(sum, p);
                            sum1 = add2(sum1, q);
                            pk[i / 2] = pack_bf16(p.x, p.y);
                            pk[i / 2 + 1] = pack_bf16(q.x, q.y);
                        }
                        tm_st16(tS + 16 * k, pk);
                    }
                    l += (sum.x + sum.y) + (sum1.x + sum1.y);
                    tm_wait_st();
                    tcf_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&nt->p_full[w]);
            }
            if (!ok) break;
            // ---- this segment's sums
            const bool whole = wk.j0 == 0 && wk.j1 == wk.T;
            const bool steps = first_j < e;
            if (steps) {
                ok = tc_wait(&nt->o_done[w], oc & 1, a.status);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                ++oc;
                tcf_after();
            }
            // One tile with two streams: stream 0 takes both sums to the result. They stand in
            // the same lanes of tensor memory.
            const bool join = !pair && wk.j1 - wk.j0 > 1;
            float m2 = m == -SPLA_INF ? -SPLA_INF : m * a.sl2, f0 = 1.f, f1 = 0.f;
            bool has0 = true, has1 = false;             // whether a stream has a part in the row
            if (join && w == 1) {
                nt->m1[r] = m2;
                nt->l1[r] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(&nt->m_full);
                ok = tc_wait(&nt->m_empty, mc & 1, a.status);
            } else if (join) {
                ok = tc_wait(&nt->m_full, mc & 1, a.status);
                const float n2 = nt->m1[r], l1 = nt->l1[r], M = fmaxf(m2, n2);
                // no tokens: no part; nothing but NaN logits: NaN; else a part whatever the
                // weight, since a weight of zero makes NaN of an infinity or NaN among the sums
                has0 = has_part(m2, l);
                has1 = has_part(n2, l1);
                f0 = m2 == -SPLA_INF ? l : ex2(m2 - M);
                f1 = n2 == -SPLA_INF ? l1 : ex2(n2 - M);
                l = (has0 ? l * f0 : 0.f) + (has1 ? l1 * f1 : 0.f);
                m2 = M;
            }
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            mc += join;
            tcf_after();
            // a unit cut by this run's end starts a partial 1 unless it began before the run
            const int slot = wk.j0 == 0 ? 1 : 0;
            float* part = reinterpret_cast<float*>(a.ws + kCutBytes) +
                          ((int64_t)blockIdx.x * 2 + slot) * part_floats(D);
            const int row = (pair ? w * 128 : 0) + r;
            if (warp_live && (pair || w == 0)) {
                const bool notes = steps && *(volatile int32_t*)&nt->nf_seg == seg;
                const float inv = 1.f / l;
                const int64_t orow = ((int64_t)(wk.b * (int64_t)a.max_new + tok) * c.hq +
                                      wk.h * G + (r & (G - 1)));
#pragma unroll 1                                        // (cold code is fetched at every launch)
                for (int i = 0; i < D; i += 32) {
                    float o[32];
                    if (steps) {
                        tm_ld32(tO + i, o);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0.f;
                    }
                    if (join) {
                        float y[32];
                        tm_ld32(tO + 128 + i, y);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = (has0 ? o[k] * f0 : 0.f) + (has1 ? y[k] * f1 : 0.f);
                    }
                    if (live && whole) {
                        uint4* d = reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + orow * D + i);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            d[k] = make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv),
                                              pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                              pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                              pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                    } else if (live) {
                        float4* d = reinterpret_cast<float4*>(part + (int64_t)row * D + i);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            d[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                    __syncwarp();                       // the next load is the whole warp's
                }
                if (notes && live) {                    // rare: infinities and NaN that were seen
                    __threadfence_block();              // the notes after their flag
#pragma unroll 1
                    for (int i = 0; i < D; ++i) {
                        const float x = note_term(nt->first[0][i], nt->first[1][i], nt->first[2][i], pos);
                        if (x == 0.f) continue;
                        if (whole) {
                            __nv_bfloat16* d = (__nv_bfloat16*)a.out + orow * D + i;
                            *d = __float2bfloat16_rn(__bfloat162float(*d) + x);
                        } else {
                            part[(int64_t)row * D + i] += x;
                        }
                    }
                    __threadfence_block();              // and before this warp is counted
                }
                if (live && whole) {
                    if (a.lse) a.lse[orow] = (m2 + log2f(l)) * 0.69314718055994531f;
                } else if (live) {
                    part[256 * D + row] = m2;
                    part[256 * D + 256 + row] = l;
                }
            }
            wk.note_cut(cut, blockIdx.x, U, G, nt->run);
            tcf_before();
            __syncwarp();
            if (join && w == 0 && lane == 0) mbar_arrive(&nt->m_empty);
            if (lane == 0) atomicAdd(&nt->epi[w], 1);      // (the notes were consumed above)
            ++seg;
        }
        if (tid == 0) reinterpret_cast<ChunkCut*>(a.ws)[blockIdx.x] = cut;
    }
    tcf_before();
    asm volatile("bar.sync 1, %0;" :: "n"(kTcThreads) : "memory");
    }
}

// ------------------------------------------------------------------ host launcher
template <int D, bool kTwo>
static cudaError_t launch_tc(const CacheView& c, const CUtensorMap& tq, const CUtensorMap& tk,
                             const CUtensorMap& tv, const ChunkArgs& a, cudaStream_t s) {
    using S = TcShape<D, kTwo>;
    // the register shares are of a launch with kTcRegs a thread: with fewer, the softmax
    // warps would wait for registers that nobody gives back
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, chunk_tc_kernel<D, kTwo>);
        if (e != cudaSuccess) return e;
        regs.store(f.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < kTcRegs) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(chunk_tc_kernel<D, kTwo>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(chunk_tc_kernel<D, kTwo>, dim3(kMaxRuns), dim3(kTcThreads), S::kSmem, s, tq, tk,
                   tv, c, a);
    if (e != cudaSuccess) return e;
    const int rows = (int)std::min<int64_t>(S::kRows, (int64_t)a.max_new * c.group);
    return launch_chunk_combine(c, SPLA_BF16, a, rows, s);
}

// tq: [batch][max_new][Hq][d] with boxes of 64 dims x G heads x 128 / G tokens; tk, tv:
// the pools as rows of d with boxes of 64 dims x 64 tokens.
cudaError_t launch_chunk_tc(const CacheView& c, const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, const ChunkArgs& a, cudaStream_t s) {
    // two query tiles need more rows than one holds; one tile then takes half the MMAs
    const bool two = (int64_t)a.max_new * c.group > 128;
    if (c.d == 128)
        return two ? launch_tc<128, true>(c, tq, tk, tv, a, s) : launch_tc<128, false>(c, tq, tk, tv, a, s);
    return two ? launch_tc<64, true>(c, tq, tk, tv, a, s) : launch_tc<64, false>(c, tq, tk, tv, a, s);
}

}  // namespace spla
