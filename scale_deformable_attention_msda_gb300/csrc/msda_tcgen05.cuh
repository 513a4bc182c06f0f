// tcgen05, TMA and mbarrier pieces (sm_103a) for kernels whose operands lie in
// swizzled tiles of shared memory and whose accumulators lie in tensor memory.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace msda {

__device__ __forceinline__ uint32_t shared_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ------------------------------------------------------------- mbarriers
// Waits are bounded: one of two seconds (they take microseconds) sets the block's
// `dead` word, whereupon every other wait of the block gives up too, and bit 1 of
// the device word. A pause between two looks at the timer, as of a process whose turn on
// the GPU was another's, counts as ten milliseconds at most: what ran out is time that the
// block had.
constexpr unsigned long long kWaitNs = 2000000000ull, kPauseNs = 10000000ull;

__device__ __forceinline__ unsigned long long nanoseconds() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// One lane of a whole warp issues the instruction, always the same one. The warp's
// code around it stays uniform, and with it descriptors and addresses, which these
// instructions take from uniform registers: an MMA of 128 x 32 x 16 with its left operand
// in tensor memory then takes 16 cycles, and 45 to 70 issued from a branch of one lane.
#define ELECT(instruction) "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t@one " instruction "\n\t}"

__device__ __forceinline__ void bar_arrive_one(uint64_t *bar) {
    asm volatile(ELECT("mbarrier.arrive.shared::cta.b64 _, [%0];") ::"r"(shared_at(bar)) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_at(bar)) : "memory");
}
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_at(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_done() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
    asm volatile(ELECT("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;") ::"r"(shared_at(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(shared_at(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}
// The rest of a wait whose first look found the phase not there. False when it ran out,
// here or in another wait of the block.
__device__ __forceinline__ bool bar_wait_more(uint64_t *bar, uint32_t parity, volatile uint32_t *dead, unsigned *err) {
    unsigned long long last = 0, waited = 0;
    for (uint32_t i = 1;; ++i) {
        if (bar_try(bar, parity)) return true;
        if (i & 63u) continue;         // the timer is slow to read
        if (*dead) return false;
        const unsigned long long now = nanoseconds();
        if (last != 0) waited += now - last < kPauseNs ? now - last : kPauseNs;
        last = now;
        if (waited > kWaitNs) break;
    }
    if (bar_try(bar, parity)) return true;
    *dead = 1u;
    if (err) atomicOr(err, 2u);
    return false;
}
// For a whole warp, whose lanes agree. A barrier's phase of the other parity than the one
// under way counts as there: so does, before the first, that of parity 1.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *dead, unsigned *err) {
    if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
    return __all_sync(0xffffffffu, bar_wait_more(bar, parity, dead, err));
}
// A barrier and the parity of the phase waited for.
struct Phase {
    uint64_t *bar;
    uint32_t parity;
};
// Waits for all of them, and looks at all before it acts on one.
template <class... P>
__device__ __forceinline__ bool bar_wait_all(volatile uint32_t *dead, unsigned *err, P... phases) {
    bool now = true;
    ((now = bar_try(phases.bar, phases.parity) && now), ...);
    if (__all_sync(0xffffffffu, now)) return true;
    bool ok = true;
    ((ok = ok && bar_wait_more(phases.bar, phases.parity, dead, err)), ...);
    return __all_sync(0xffffffffu, ok);
}
// Place and phase in a ring of N.
template <int N> struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1u;
        }
    }
};

// What this thread wrote to shared memory is there for the MMAs that follow.
__device__ __forceinline__ void shared_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A group of four warps gives registers back, or takes them: what the block was launched
// with is enough for all.
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// ------------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_load(void *to, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(ELECT("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];")
                 ::"r"(shared_at(to)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(shared_at(bar))
                 : "memory");
}
// `bytes`, a multiple of 16, from and to 16-byte boundaries.
__device__ __forceinline__ void bulk_load(void *to, const void *from, uint32_t bytes, uint64_t *bar) {
    asm volatile(ELECT("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];")
                 ::"r"(shared_at(to)), "l"(from), "r"(bytes), "r"(shared_at(bar))
                 : "memory");
}

// ---------------------------------------------------------- tensor memory
template <int COLS> __device__ __forceinline__ void tmem_alloc(uint32_t *slot) {   // one warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_at(slot)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS> __device__ __forceinline__ void tmem_free(uint32_t at) {       // the same warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "n"(COLS));
}
__device__ __forceinline__ void tmem_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// N columns of the calling warp's 32 lanes, one lane's row to each thread. The wait is in
// the same statement, so that nothing is done with the registers before it.
#define TMEM_OUT8(o) "=&r"(v[o]), "=&r"(v[o + 1]), "=&r"(v[o + 2]), "=&r"(v[o + 3]), "=&r"(v[o + 4]), "=&r"(v[o + 5]), "=&r"(v[o + 6]), "=&r"(v[o + 7])
#define TMEM_OUT32(o) TMEM_OUT8(o), TMEM_OUT8(o + 8), TMEM_OUT8(o + 16), TMEM_OUT8(o + 24)
#define TMEM_R0 "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
#define TMEM_R1 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
#define TMEM_R2 "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47"
#define TMEM_R3 "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
#define TMEM_R4 "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79"
#define TMEM_R5 "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95"
#define TMEM_R6 "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111"
#define TMEM_R7 "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127"
#define TMEM_WAIT "tcgen05.wait::ld.sync.aligned;"
template <int N> __device__ __forceinline__ void tmem_read(uint32_t (&v)[N], uint32_t at);
template <> __device__ __forceinline__ void tmem_read<16>(uint32_t (&v)[16], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {" TMEM_R0 "}, [%16];\n\t" TMEM_WAIT
                 : TMEM_OUT8(0), TMEM_OUT8(8) : "r"(at) : "memory");
}
template <> __device__ __forceinline__ void tmem_read<32>(uint32_t (&v)[32], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {" TMEM_R0 "," TMEM_R1 "}, [%32];\n\t" TMEM_WAIT
                 : TMEM_OUT32(0) : "r"(at) : "memory");
}
template <> __device__ __forceinline__ void tmem_read<64>(uint32_t (&v)[64], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {" TMEM_R0 "," TMEM_R1 "," TMEM_R2 "," TMEM_R3 "}, [%64];\n\t" TMEM_WAIT
                 : TMEM_OUT32(0), TMEM_OUT32(32) : "r"(at) : "memory");
}
template <> __device__ __forceinline__ void tmem_read<128>(uint32_t (&v)[128], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {" TMEM_R0 "," TMEM_R1 "," TMEM_R2 "," TMEM_R3 "}, [%128];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x64.b32 {" TMEM_R4 "," TMEM_R5 "," TMEM_R6 "," TMEM_R7 "}, [%129];\n\t" TMEM_WAIT
                 : TMEM_OUT32(0), TMEM_OUT32(32), TMEM_OUT32(64), TMEM_OUT32(96) : "r"(at), "r"(at + 64) : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// Two ranges of N columns each.
template <int N> __device__ __forceinline__ void tmem_read_two(uint32_t (&v)[N], uint32_t (&w)[N], uint32_t at, uint32_t at2);
#define TMEM_OUT8W(o) "=&r"(w[o]), "=&r"(w[o + 1]), "=&r"(w[o + 2]), "=&r"(w[o + 3]), "=&r"(w[o + 4]), "=&r"(w[o + 5]), "=&r"(w[o + 6]), "=&r"(w[o + 7])
#define TMEM_OUT32W(o) TMEM_OUT8W(o), TMEM_OUT8W(o + 8), TMEM_OUT8W(o + 16), TMEM_OUT8W(o + 24)
template <> __device__ __forceinline__ void tmem_read_two<64>(uint32_t (&v)[64], uint32_t (&w)[64], uint32_t at, uint32_t at2) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {" TMEM_R0 "," TMEM_R1 "," TMEM_R2 "," TMEM_R3 "}, [%128];\n\t"
                 "tcgen05.ld.sync.aligned.32x32b.x64.b32 {" TMEM_R4 "," TMEM_R5 "," TMEM_R6 "," TMEM_R7 "}, [%129];\n\t" TMEM_WAIT
                 : TMEM_OUT32(0), TMEM_OUT32(32), TMEM_OUT32W(0), TMEM_OUT32W(32) : "r"(at), "r"(at2) : "memory");
}
template <int N> __device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&v)[N]);
#define TMEM_IN8(o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
#define TMEM_IN32(o) TMEM_IN8(o), TMEM_IN8(o + 8), TMEM_IN8(o + 16), TMEM_IN8(o + 24)
template <> __device__ __forceinline__ void tmem_store<32>(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {" TMEM_R0 "," TMEM_R1 "};" ::TMEM_IN32(0), "r"(at) : "memory");
}

// ------------------------------------------------------------------- MMA
// A tile of rows of 64 or 128 bytes as TMA writes it with the swizzle of that
// width. PITCH: bytes of a row. Rows lie in groups of 8; a tile wider than 128
// bytes is several such panels.
//
// Read along the rows' contents (K-major: the contraction runs within a row), the
// descriptor's stride is that of a group of 8 rows. Read across them (MN-major:
// the contraction runs over the rows), it is the same stride between 8 steps of
// the contraction, and the leading stride is that of a panel.
//
// The descriptor's two words: the low one has the address and the leading stride, and
// a step along the tile adds to it (offset / 16); the high one is constant.
__device__ __forceinline__ constexpr uint32_t desc_step(uint32_t bytes) { return bytes >> 4; }
__device__ __forceinline__ uint32_t desc_low(uint32_t at, uint32_t panel_bytes) {
    return ((at & 0x3ffffu) >> 4) | ((panel_bytes >> 4) << 16);
}
template <int PITCH> __device__ __forceinline__ constexpr uint32_t desc_high() {
    static_assert(PITCH == 64 || PITCH == 128, "the tile's swizzle");
    return (uint32_t)(8 * PITCH >> 4) | (1u << 14) | ((PITCH == 128 ? 2u : 4u) << 29);
}
// No swizzle: runs of 16 bytes, 8 rows' together; the leading stride is that of the next
// run of the same rows, the other one that of the next 8 rows.
__device__ __forceinline__ constexpr uint32_t desc_high_plain(uint32_t group_bytes) { return (group_bytes >> 4) | (1u << 14); }
// fp32 accumulators of 16-bit operands (bf16, or fp16), 128 rows by N columns.
template <bool BF16, int N, bool B_ACROSS>
__device__ __forceinline__ constexpr uint32_t mma_desc() {
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((B_ACROSS ? 1u : 0u) << 16) |
           ((uint32_t)(N / 8) << 17) | ((uint32_t)(128 / 16) << 24);
}
// d (+)= a b' of descriptors with the same high word; idesc and high are constants.
template <uint32_t IDESC, uint32_t HIGH>
__device__ __forceinline__ void mma_shared(uint32_t d, uint32_t a, uint32_t b, bool add) {
    asm volatile("{\n\t.reg .pred p, one;\n\t.reg .b64 da, db;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                 "@one tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"((uint32_t)add), "n"(IDESC), "n"(HIGH)
                 : "memory");
}
template <uint32_t IDESC, uint32_t HIGH>
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, bool add) {
    asm volatile("{\n\t.reg .pred p, one;\n\t.reg .b64 db;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "mov.b64 db, {%2, %5};\n\t"
                 "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"((uint32_t)add), "n"(IDESC), "n"(HIGH)
                 : "memory");
}
// Arrives at `bar` when every MMA issued before has finished.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile(ELECT("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];") ::"r"(shared_at(bar)) : "memory");
}

}  // namespace msda
