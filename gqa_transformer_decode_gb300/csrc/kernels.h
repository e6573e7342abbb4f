// kernels.h -- launch interfaces of the ember kernels (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ember.h"

namespace ember {

// Host-side count of kernel launches (every launch_* call adds its kernels).
void count_launches(long long n);
// Records an event before the launch of kernel fn when the calling thread
// traces a decode step (ember_decode_step_traced); otherwise does nothing.
void trace_launch(const void* fn, cudaStream_t s);
unsigned long long launches_so_far();
// Sets the calling thread's ember_last_error message and returns st.
ember_status set_error(ember_status st, const char* fmt, ...);

// Launch with the programmatic-stream-serialization attribute (PDL) unless
// disabled (EMBER_NO_PDL=1): the kernel may start while its predecessor in
// the stream finishes, and must pdl_wait() before reading its outputs.
bool pdl_enabled();
template <typename... KArgs, typename... Args>
inline cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t s, Args&&... args) {
    count_launches(1);
    trace_launch(reinterpret_cast<const void*>(kern), s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// The same with the grid's x dimension in thread-block clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                                    cudaStream_t s, Args&&... args) {
    count_launches(1);
    trace_launch(reinterpret_cast<const void*>(kern), s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Runs f, a setting of a kernel's, for the current device unless it has succeeded there before
// (0.3 us a call otherwise).
class OncePerDevice {
    std::atomic<uint64_t> done_{0};

public:
    template <class F>
    cudaError_t operator()(F f) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = f();
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// ---------------------------------------------------------------- embedding --
// x[t] = f32(E[ids[t]]) and the per-token argument checks of a decode step
// (seq in range, position == cursor, position < max_len, id < vocab) or of a
// prefill (start position == cursor).
struct EmbedArgs {
    const uint16_t* E;
    int V, H;
    const int32_t* ids;
    int n;
    float* x;                    // [n][H]
    int* status;
    // decode-step checks (seqs == nullptr for prefill / encode)
    const int32_t* seqs;
    const int32_t* positions;
    const int32_t* cursor;
    int max_seqs, max_len;
    int* tok_ok;                 // [n] 1 = token may touch the cache
    int32_t* tok_pos;            // [n] resolved position (positions[t] or the cursor)
    // prefill check (pf_seq < 0: none)
    int pf_seq, pf_start;
    float* zero0;                // [n][zlen] set to 0 when non-null (residual accumulators)
    float* zero1;
    int zlen;                    // floats per token zeroed in zero0 / zero1 (0: H)
};
void launch_embed(const EmbedArgs& a, cudaStream_t s);

// --------------------------------------------------------------------- GEMV --
// Batch-1..8 decode projections: y[b][n] = rinv_b * sum_k W[n][k] x[b][k] w_k
// with the RMSNorm of x fused into the prologue when norm_w != nullptr.
struct GemvArgs {
    const uint16_t* W;           // [N][K] bf16, or f16 when w_f16 (unused when Wq is set)
    int N, K;
    int w_f16;
    const int8_t* Wq;            // q8_0 weights: codes [N][K] (K % 32 == 0), or nullptr
    const uint16_t* Wd;          // q8_0 scales [N][K/32] (f16 bits)
    const float* x;              // [nb][ldx] f32
    int ldx;
    const float* norm_w;         // [K] f32 or nullptr
    float eps;
    const float* bias;           // [N] f32 or nullptr (EPI_STORE)
    float* out;                  // mode-dependent, row stride ldo
    int ldo;
    int nb;
    int mode;                    // EpiMode
    unsigned long long* keys;    // [nb] argmax keys (EPI_ARGMAX)
    int* status;
    int w_exp;                   // W stored scaled by 2^-w_exp: products multiplied by 2^w_exp
    const float* x_add;          // [x_add_slots][K] summed into x (split-K accumulator copies;
                                 // nb == 1, bf16 W), or nullptr
    int x_add_slots;
};
// Returns the launch's own error (not the thread's pending last error).
cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t s, int num_sms);

// ------------------------------------------------------- decode attention --
// Split-KV flash decoding: one CTA per (token, kv head, split), all G query
// heads of the kv head together; the last CTA of a (token, kv head) merges the
// splits.  Also applies q/k norm + RoPE and writes the token's K/V row.
struct AttnDecodeArgs {
    const float* qkv;            // [nb][ld_qkv] pre-RoPE q | k | v (biased)
    int ld_qkv;
    int nb, NH, NKV, D, L, layer;
    const int32_t* seqs;
    const int32_t* positions;    // resolved positions (the embed kernel's tok_pos)
    const int* tok_ok;
    uint16_t* kc;                // K cache base [S][L][NKV][max_len][D]
    uint16_t* vc;
    int max_len;
    const float* cos_t;          // [max_len][D/2]
    const float* sin_t;
    const float* q_norm;         // [D] or nullptr
    const float* k_norm;
    float eps;
    float* att;                  // [nb][NH*D] f32 (used when att_b == nullptr)
    uint16_t* att_b;             // [nb][NH*D] f16 GEMM operand, or nullptr
    float* part;                 // split partials
    unsigned* counters;          // [nb*NKV], zero between launches
    int splits;
    int* status;
    const void* k_map;           // host copies of the caches' 3-D TMA maps, or nullptr
    const void* v_map;           // (read by the launcher only)
};
void launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t s);
// The same on the warp tensor cores (decode_attn_mma.cu): head_dim 64 / 128,
// at most 16 query heads per kv head, K/V through the TMA maps.
// launch_attn_decode picks it when the maps are given.
bool attn_decode_mma_supported(int D, int G);
void launch_attn_decode_mma(const AttnDecodeArgs& a, cudaStream_t s);

// Greedy argmax write-back and cursor advance at the end of a step.
struct FinishArgs {
    int nb;
    unsigned long long* keys;    // reset to 0 here
    int32_t* argmax;             // [nb] or nullptr
    // decode: cursor[seqs[b]] = positions[b] + 1 for ok tokens
    const int32_t* seqs;
    const int32_t* positions;
    const int* tok_ok;
    int32_t* cursor;
    // prefill: cursor[pf_seq] = pf_end (pf_seq >= 0)
    int pf_seq, pf_end;
};
void launch_finish(const FinishArgs& a, cudaStream_t s);
void launch_set_cursor(int32_t* cursor, int seq, int pos, cudaStream_t s);

// ------------------------------------------------------------- prefill side --
// xb[t] = f16(RMSNorm(x[t]) * w)   (A operand of the tensor-core GEMMs);
// with zero set, also zero[t][0, zlen) = 0 (the next GEMM's split-K output)
void launch_rmsnorm_h(const float* x, const float* w, float eps, int n, int H, uint16_t* xb,
                      int* status, cudaStream_t s, float* zero = nullptr, int zlen = 0);
// xb[t] = bf16(RMSNorm(x[t]) * w)   (A operand of the tied-head GEMM)
void launch_rmsnorm_bf16(const float* x, const float* w, float eps, int n, int H, uint16_t* xb,
                         cudaStream_t s);
// h[t] = RMSNorm(x[t]) * w  in f32
void launch_rmsnorm_f32(const float* x, const float* w, float eps, int n, int H, float* h,
                        cudaStream_t s);

// q/k norm + RoPE of n tokens; q -> bf16 [n][NH*D]; K, V rows -> bf16 cache.
// Token t of sequence z = t / T_per_seq goes to position pos0 + t % T_per_seq
// of cache rows k + z*seq_stride + g*head_stride + pos*D.
struct RopeKVArgs {
    const float* qkv;
    int ld_qkv;
    int n, NH, NKV, D;
    int T_per_seq, pos0;
    const float* cos_t;
    const float* sin_t;
    const float* q_norm;
    const float* k_norm;
    float eps;
    uint16_t* q_out;             // [n][NH*D] f16 (the attention MMA operand)
    uint16_t* kc;
    uint16_t* vc;
    long long seq_stride, head_stride;
    // nullable: the f16 copy of each new K row (the value the bf16 cache
    // holds) also goes to kh[(z * NKV + g) * kh_pad + pos][D], the tensor-core
    // attention's K operand
    uint16_t* kh;
    int kh_pad;
};
void launch_rope_kv(const RopeKVArgs& a, cudaStream_t s);

// Whole-prompt attention reading K/V rows from the cache layout above.
// Query row t of sequence z sits at position pos0 + t; keys [0, pos0+t] are
// visible when causal, [0, T_per_seq + pos0) otherwise.
struct AttnPrefillArgs {
    const uint16_t* q;           // [n][NH*D] f16, RoPE'd
    int n, NH, NKV, D;
    int T_per_seq, pos0, causal;
    const uint16_t* kc;
    const uint16_t* vc;
    long long seq_stride, head_stride;
    uint16_t* att;               // [n][NH*D] f16 (GEMM operand)
    int* status;
};
void launch_attn_prefill(const AttnPrefillArgs& a, cudaStream_t s);

// out[t][j] = sum_k h[t][k] W[j][k] + b[j]  (label head, f32 h)
void launch_cls_head(const float* h, int n, int H, const uint16_t* W, const float* b, int labels,
                     float* out, cudaStream_t s);

// out[b][j] = mean_t h[b*T + t] . W[j] + bias[j] (mean-pooled head; bf16 W, bias)
cudaError_t launch_pooled_head(const float* h, int B, int T, int H, const uint16_t* W, const uint16_t* b,
                               int n_out, float* out, cudaStream_t s);
// dst[0..n) = src[0..n) (f32), ordered after the previous kernel
void launch_copy_f32(float* dst, const float* src, int n, cudaStream_t s);

// Standalone RoPE + bf16 store (kernel-level parity entry point).
void launch_rope_store(const float* x, int n_tok, int n_heads, int D, const float* cos_t,
                       const float* sin_t, uint16_t* out, cudaStream_t s);

// bf16 [n] -> f32 [n] (weight repack of norms / biases)
void launch_bf16_to_f32(const uint16_t* in, float* out, long long n, cudaStream_t s);
// bf16 bits -> f16 bits in place (weight repack of the layer matrices)
// q8_0 quantization of n bf16 values at p (n % 32 == 0): codes q[n], f16
// scales d[n/32]; f16_out (nullable, may be p) receives the f16 of the
// decoded values times 2^-f16_exp.
void launch_q8_0_quantize(const uint16_t* p, long long n, int8_t* q, uint16_t* d, uint16_t* f16_out,
                          int f16_exp, cudaStream_t s);
void launch_bf16_to_f16_inplace(uint16_t* p, long long n, int exp, cudaStream_t s);
// *out = max(*out, max |p[i]|) as f32 bits, over n bf16 values (NaN skipped)
void launch_absmax_bf16(const uint16_t* p, long long n, unsigned* out, cudaStream_t s);

// ----------------------------------------------------------- tcgen05 GEMM --
// D[M,N] = A[M,K] . B[N,K]^T (bf16 in, f32 accumulate in TMEM) with a fused
// epilogue.  A and B are described by TMA tensor maps made by make_gemm_plan.
struct GemmEpilogue {
    int mode;                    // EpiMode (EPI_STORE, EPI_RESID, EPI_SWIGLU, EPI_ARGMAX)
    float* out_f32;              // EPI_STORE / EPI_RESID: [M][ldo]; EPI_ARGMAX: logits or nullptr
    uint16_t* out_h;             // EPI_SWIGLU: [M][ldo] f16 (N/2 columns)
    int ldo;
    const float* bias;           // EPI_STORE, nullable
    unsigned long long* keys;    // EPI_ARGMAX: [M] argmax keys (start at 0)
    int ksplit;                  // set by launch_gemm: K split over grid.z (red.add outputs)
    int w_exp;                   // B is stored scaled by 2^-w_exp: products are multiplied by 2^w_exp
    int zeroed;                  // EPI_STORE: out_f32 is zero, so K may be split
    // Host pointer to a tensor map over the output (make_out_map), or null.
    // The many-row GEMM then writes its EPI_STORE / EPI_RESID / EPI_SWIGLU
    // tiles through shared memory with TMA (EPI_RESID as an f32 reduce-add);
    // the map's rows bound the rows written.
    const void* out_map;
};
// Tensor map over an output [rows][ld] (cols <= ld) for GemmEpilogue.out_map:
// f32 with 32 x 128 boxes, or f16 (the SwiGLU output) with 64 x 128 boxes,
// 128-byte swizzle.  False if the driver rejects it.
bool make_out_map(void* out, const void* ptr, int rows, int cols, int ld, bool f16);

struct GemmPlan {
    alignas(64) unsigned char tmA[128];
    alignas(64) unsigned char tmB[128];
    alignas(64) unsigned char tmB64[128];   // B with a 64-row box (few-row A, split-K)
    int M, N, K;
    int bn;                      // N tile (64, 128 or 256)
    int sms;                     // SMs of the device the plan was made on
    bool f16;                    // operands f16 (else bf16)
    bool ok;
};
// A rows = M (activations), B rows = N (weights); both row-major with K
// contiguous and 16-byte aligned rows.  Returns false if the driver rejects
// the tensor maps.
bool make_gemm_plan(GemmPlan& p, const uint16_t* A, int M, int lda, const uint16_t* B, int N,
                    int ldb, int K, bool f16);
// For m_rows <= 128 (one row tile) the GEMM runs with 64-column tiles and,
// for EPI_STORE / EPI_RESID, splits K across CTAs until about one CTA per SM;
// the partial sums are added with red.global.add, so EPI_STORE then needs a
// zeroed output.  gemm_splits() returns the split launch_gemm will use.
int gemm_splits(const GemmPlan& p, int m_rows, int mode);
// Persistent tiles for m_rows > 128 (gemm_persistent.cu); launch_gemm picks it.
void launch_gemm_persistent(const void* tmA, const void* tmB, int bn, int m_rows, int N, int K,
                            uint32_t idesc, const GemmEpilogue& e, int* status, int sms,
                            cudaStream_t s);
// Encode a bf16 TMA tensor map (rank 2..4, 128-byte swizzle, zero fill out
// of bounds).  dims[0] is the contiguous dimension; strides (rank-1 entries)
// are in bytes.  False if the driver rejects it.
bool encode_map_bf16(void* out, const void* ptr, int rank, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box);
// The same with the 32-byte swizzle (boxes of 16 elements a row).
bool encode_map_bf16_sw32(void* out, const void* ptr, int rank, const uint64_t* dims,
                          const uint64_t* strides, const uint32_t* box);
// Rows of f32 or 16-bit elements, ld apart, not swizzled.
bool encode_map_rows(void* out, const void* ptr, bool f32, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_cols,
                     uint32_t box_rows);

// m_rows: rows of A actually valid (<= p.M); the rest is ignored.
void launch_gemm(const GemmPlan& p, int m_rows, const GemmEpilogue& e, int* status,
                 cudaStream_t s);

// ------------------------------------------------ tensor-core attention --
// Whole-prompt GQA attention on tcgen05 (head_dim 64 or 128).  Maps: Q over
// the f16 queries [rows][NH*D] (box 64 x 128); K over the f16 copy of the K
// rows Kh [z][keys_pad][D] (3-D, box 64 x 128 x 1); Vt over transposed f16 V
// [z][D][keys_pad] (3-D, box 64 x D x 1).  Query row t of sequence z
// (t < T_per_seq) sits at position pos0 + t; it reads Kh and Vt at z index
// z*NKV + g.
struct AttnTcArgs {
    int T_per_seq, pos0, causal, n_keys;
    int NH, NKV, G;
    uint16_t* att;               // [rows][ld_att] f16 (GEMM operand)
    int ld_att;
    int* status;
};
bool attn_tc_supported(int D);
void launch_attn_tc(const void* map_q, const void* map_k, const void* map_vt, const AttnTcArgs& a,
                    int nseq, int D, cudaStream_t s);
// head_dim 64 / 128, two query tiles per CTA in ping-pong (attn_tc2.cu)
void launch_attn_tc2(const void* map_q, const void* map_k, const void* map_vt, const AttnTcArgs& a,
                     int nseq, int D, cudaStream_t s);

// Vt[z][d][key] = f16(V[z][key][d]) and Kh[z][key][d] = f16(K[z][key][d]) for
// keys < n_keys, 0 for keys in [n_keys, keys_pad): V (and K) rows of index
// z = (z / nkv, z % nkv) start at v + (z/nkv)*v_z_stride + (z%nkv)*v_h_stride
// (the same offsets from k).  kh may be null; Kh rows in [kh_from, n_keys)
// are left alone (the RoPE kernel wrote them).
struct VtArgs {
    const uint16_t *v, *k;
    long long v_z_stride, v_h_stride;
    int nkv, D, n_keys, keys_pad;
    uint16_t *vt, *kh;
    int kh_from;
};
void launch_vt(const VtArgs& a, int zs, cudaStream_t s);

// ------------------------------------------- fused batch-1 decode layer --
// Two kernels per decoder layer (decode_fused.cu).  Residual stream of kernel
// n: x_n = x_in + z_in; the kernel writes x_out = x_n, zeroes z_zero and adds
// its output into z_acc (three rotating accumulators, two x buffers).
// The batch-1 decode's split-K accumulators have ZSLOTS copies of the
// hidden vector: a CTA adds into copy (CTA index % ZSLOTS) and a reader sums
// the copies, so that ZSLOTS times fewer atomic additions meet at one address.
constexpr int ZSLOTS = 8;

struct FusedPlan {
    int C = 0;           // CTAs per cluster (one cluster per kv head)
    int nr = 0, no = 0;  // q/k/v rows and o_proj rows per CTA
    int smem_attn = 0, smem_mlp = 0;
    int ns = 0;          // weight ring stages of the MLP kernel
    int fc = 0;          // intermediate features per MLP chunk (4, 8 or 16)
    int xi = 0;          // 16-byte input chunks per lane in the row dots (4: inputs <= 1024, 8: <= 2048)
    int mlp_grid = 0;
    bool resident = false;   // every MLP CTA's chunks fit its shared memory (ns = chunks per CTA)
    bool part = false;       // partitioned: attention and MLP blocks on disjoint SMs, all weights resident
    int zs = ZSLOTS;         // copies of the MLP block's split-K accumulator (1..ZSLOTS)
    int mlp_delay_ns = 0;    // partitioned: MLP weight copies start this long after the CTA arrives
    int pf_late = 0;         // MLP CTAs that start after the attention (their chunks are prefetched to L2)
    bool ok = false;
    const char* why = "not planned";   // reason when !ok
};
bool fused_decode_plan(FusedPlan& p, int H, int NH, int NKV, int D, int F, int num_sms);

struct FusedAttnArgs {
    const uint16_t* wqkv;        // f16 [q rows | k rows | v rows][H]
    const float* bqkv;           // or nullptr
    const float* norm_w;
    float eps;
    const float* q_norm;         // [D] or nullptr (then k_norm unused)
    const float* k_norm;
    const uint16_t* wo;          // f16 o_proj grouped by kv head: [NKV][H][G*D]
    int H, NH, NKV, D, L, layer;
    const float* x_in;
    const float* z_in;
    float* x_out;
    float* z_zero;
    float* z_acc;
    uint16_t* kc;                // K / V cache [seq][layer][kv head][max_len][D] bf16
    uint16_t* vc;
    int max_len, max_seqs;
    const int32_t* seqs;
    const int32_t* tok_pos;
    const int* tok_ok;
    const int32_t* positions;    // the step's explicit positions (nullptr: the cursor)
    const int32_t* cursor;       // [max_seqs] the cache's cursors
    int resident;                // resident plan: o_proj rows and two K/V tiles loaded before the wait
    int qkv_exp, o_exp;          // storage scales of wqkv / wo (2^-e), undone on the products
    int zs;                      // accumulator copies the MLP block before this one added into
    const float* cos_t;
    const float* sin_t;
    int* status;
    int C, nr, no;
};
// k_map / v_map: 3-D TMA maps (D, max_len, seqs*layers*kv heads), box 64 x 128 x 1
void launch_fused_attn(const void* k_map, const void* v_map, const FusedAttnArgs& a, int xi, int smem,
                       cudaStream_t s);

struct FusedMlpArgs {
    const uint16_t* wgu;         // f16 [2F][H], row 2f gate_f, row 2f+1 up_f
    const uint16_t* wdT;         // f16 [F][H] (down_proj transposed)
    const float* norm_w;
    float eps;
    int H, F;
    const float* x_in;
    const float* z_in;
    float* x_out;
    float* z_zero;
    float* z_acc;
    int* status;
    int ns;
    int pf_late;                 // the last pf_late CTAs start late: the others prefetch their chunks to L2
    int load_delay_ns;           // partitioned plan: delay of the weight copies after the CTA arrives
    int gu_exp, d_exp;           // storage scales of wgu / wdT (2^-e), undone on the products
    int zs;                      // accumulator copies to add into (CTA index % zs)
};
void launch_fused_mlp(const FusedMlpArgs& a, int fc, int xi, int grid, int smem, cudaStream_t s);
// One bounded mbarrier wait that nothing completes (which: 0 the CTA wait,
// 1 the cluster-scope wait), raising EMBER_ERR_TIMEOUT into status.
void launch_wait_probe(int which, long long budget, int* status, cudaStream_t s);
// The partitioned plan's MLP block: grid CTAs of 512 threads on their own SMs.
void launch_fused_mlp_res(const FusedMlpArgs& a, int xi, int grid, int smem, cudaStream_t s);

// ---------------------------------------------------------------- sampler --
// One token per row of logits [B][ldl] (V used): temperature t (t <= 0:
// greedy), top-k (0 < k < V), top-p (0 < p < 1), softmax, inverse-CDF draw
// with r[b] in [0, 1).  sampler.cu.
struct SampleArgs {
    const float* logits;
    int B, V;
    long long ldl;
    float t;
    int k;
    float p;
    const float* r;
    int32_t* out;
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- adapters --
// y = W x + bias + s_a B_a (A_a x) for each row x of a batch, a = ids[row]
// (negative: none).  adapters.cu.
struct AdapterArgs {
    const int32_t* ids;          // [n]
    int n, N, K, R, n_adapters;
    const float* scale;          // [n_adapters] or nullptr (1)
    const uint16_t* bias;        // [N] or nullptr
    const uint16_t *x, *w, *lb;  // [n][ld_x], [N][K], [n_adapters][N][R]
    long long ld_x;
    uint16_t* t;                 // [n][R / 16 rounded up][2][16]: s_a A_a x in two terms
    void* out;                   // [n][ld_out], f32 or x's type
    long long ld_out;
    int out_f32;
    int* status;
    // set by launch_adapter:
    int nt, row_tiles, col_tiles, splits;
};
// How a call is split: rows of x in a tile, tiles, CTAs of a cluster (splits: of the second
// launch they share a tile's K) and the grid, of the second launch and of the first (low_;
// low_grid 0: row by row).
struct AdapterPlan {
    int nt, row_tiles, col_tiles, splits, grid;
    bool fold, low_fold;         // accumulators are added up every AD_FOLD blocks of K
    int low_nt, low_row_tiles, low_splits, low_grid;
};
struct AdapterMaps {
    alignas(64) unsigned char w[128], x[128], x_low[128], a[128], b[128], out[128];
};
struct AdapterRows {
    const uint16_t *x, *w, *a, *b;   // [n][ld_x], [N][K], [n_adapters][R][K], [n_adapters][N][R]
    long long ld_x;
};
AdapterPlan adapter_plan(int n, int N, int K, int R, int n_adapters, bool out_f32, int sms);
size_t adapter_ws(int n, int R);
bool adapter_maps(const AdapterArgs& a, const AdapterPlan& p, const AdapterRows& r, AdapterMaps& m);
cudaError_t launch_adapter(const AdapterMaps& m, const AdapterArgs& a, const AdapterPlan& p, const AdapterRows& r, bool bf16,
                           cudaStream_t s);

// ------------------------------------------------------- log probabilities --
// Per row of logits [n][ldl] (V used) at temperature t: the given token's log
// probability and rank, the entropy, the `top` largest logits.  logprobs.cu.
struct LogprobsArgs {
    const void* logits;
    int dtype;                   // ember_dtype
    int n, V;
    long long ldl;
    float t;
    const int32_t* ids;          // [n] or nullptr
    int top;
    float* logprob;              // [n] or nullptr
    int32_t* rank;               // [n] or nullptr
    float* entropy;              // [n] or nullptr
    int32_t* top_ids;            // [n][top]
    float* top_logprobs;
    int cluster;                 // set by launch_logprobs: CTAs of a row
};
cudaError_t launch_logprobs(const LogprobsArgs& a, int sms, cudaStream_t s);

// ------------------------------------------------------------ paged cache --
// A pool of K/V pages shared by many sequences (paged_*.cu).  Row r of page p
// of kv head g starts at k + p*page_stride + g*head_stride + r*row_stride
// (elements; the same offsets from v); table[seq][i] is the page that holds
// the sequence's positions [i * page_size, (i + 1) * page_size).
struct PagedView {
    uint16_t *k, *v;
    const int32_t* table;
    int n_pages, page_shift, NKV, D, n_seqs, width;
    long long page_stride, head_stride, row_stride;
    bool bf16;                   // element type: bf16, else f16
};

// Per-head RMSNorm (optional) and RoPE of q and k, rounding, and the store of
// the K/V rows into their pages.  src: 0 f32, 1 bf16, 2 f16.
struct PagedAppendArgs {
    PagedView c;
    const void *q, *k, *v;       // [n] rows of NH*D / NKV*D / NKV*D elements (q may be null)
    int src;
    long long ld_q, ld_k, ld_v;
    int n, NH;
    const int32_t *seqs, *positions;
    const uint16_t *q_norm, *k_norm;   // [D] bf16 bits, or nullptr
    float eps;
    const float *cos_t, *sin_t;  // [n_pos][D/2]
    int n_pos;
    uint16_t* q_out;             // [n][ld_out]
    long long ld_out;
    int* status;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);

// Attention of one query token per sequence (its last position) over the
// paged cache.
struct PagedDecodeArgs {
    PagedView c;
    const uint16_t* q;           // [B][ld_q], NH*D used
    long long ld_q;
    int B, NH;
    const int32_t* seqs;         // [B] rows of the table, or nullptr (row b)
    const int32_t* lens;         // [B] keys of the sequence, the query's own among them
    int window, sinks;
    float scale;
    uint16_t* out;               // [B][ld_out]
    long long ld_out;
    float* lse;                  // [B][NH] or nullptr
    float* ws;                   // records and partials, paged_decode_ws bytes
    int* status;
    // shared prefixes (groups nullptr: none): rows groups[i] .. groups[i + 1] - 1 read keys
    // below shared[i] from table row prefixes[i]; no window then
    const int32_t *groups, *shared, *prefixes;
    int n_groups;
    // set by launch_paged_decode:
    int split;                   // CTAs that share a long sequence in cluster form
    int by_pair;                 // records stand by (sequence, kv head)
    const float* prefix;         // PagedSharedWs, to be joined
    int prefix_head, prefix_slots, prefix_rows;
};
// bytes of ws that the call's split needs (a window only ever lowers them)
size_t paged_decode_ws(const PagedView& c, int B, int NH, int window, int sinks, int sms);
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int sms, cudaStream_t s);
// The same of a call with shared prefixes (paged_shared.cu).
size_t paged_decode_shared_ws(const PagedView& c, int B, int NH, int n_groups, int sms);
cudaError_t launch_paged_decode_shared(PagedDecodeArgs a, int sms, cudaStream_t s);

// Attention of the last cu[b + 1] - cu[b] positions of each sequence.
struct PagedPrefillArgs {
    PagedView c;
    const uint16_t* q;           // [n][ld_q]
    long long ld_q;
    int n, B, NH;
    const int32_t* seqs;
    const int32_t* cu;           // [B + 1] first query row of each sequence
    const int32_t* lens;
    int window, sinks;
    float scale;
    uint16_t* out;
    long long ld_out;
    float* lse;                  // [n][NH] or nullptr
    int* status;
    int parts;                   // set by launch_paged_prefill_tc: CTAs that share a tile pair's keys
    // shared prefixes (launch_paged_shared): B groups of rows cu[g] .. cu[g + 1] - 1 read
    // shared[g] keys of table row seqs[g], row i at most lens[i] of them; no out
    const int32_t* shared;
    float* ws;                   // PagedSharedWs
    int ws_head, slots;
};
cudaError_t launch_paged_prefill(const PagedPrefillArgs& a, int sms, cudaStream_t s);
// The same on tcgen05 (paged_prefill_tc.cu; scale > 0), through TMA maps over the
// queries and the pages (paged_prefill_maps; false if the driver rejects one).
// launch_paged_prefill picks it for calls with rows enough.
struct PagedPrefillMaps {
    alignas(64) unsigned char q[128], k[128], v[128];
};
bool paged_prefill_maps(const PagedPrefillArgs& a, PagedPrefillMaps& m);
cudaError_t launch_paged_prefill_tc(const PagedPrefillArgs& a, const PagedPrefillMaps& m, int sms, cudaStream_t s);

// The partials that launch_paged_shared leaves: `head` floats (int2 {tiles of a CTA, tiles of
// all}, then for each group {its first slot, its first tile}), [slots][G][D] sums, and
// [slots][G] {m, l}.  A pair holds rows_per_pair rows of a group at most, for one kv head; pairs
// of a group stand by kv head, then by rows, each with ceil(shared / 64) tiles, and a row has
// a slot for each kv head in that order.  What CTA c has of a row lies rows_per_pair * c slots
// further.
struct PagedSharedWs {
    int head, slots, rows_per_pair;
    size_t floats;
};
PagedSharedWs paged_shared_ws(int B, int n_groups, int NH, int NKV, int D, int sms);
cudaError_t launch_paged_shared(const PagedPrefillArgs& a, const PagedPrefillMaps& m, int sms, cudaStream_t s);

// out[c][r] = in[r][c] for 16-bit elements
void launch_transpose16(const uint16_t* in, uint16_t* out, int rows, int cols, cudaStream_t s);

}  // namespace ember
