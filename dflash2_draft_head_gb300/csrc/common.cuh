// Internal declarations shared by the kernel translation units and the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace df2 {

// Longest time one on-chip wait may take before a kernel gives up (200 ms).
constexpr uint64_t kWaitNs = 200ull * 1000 * 1000;

struct DynconvArgs {
    const void* x;
    const void* hist;
    const void* base;
    const void* delta;
    void* out;
    int S, n, C, T, G;
    int in_bf16, out_bf16;
};

struct ProjectArgs {
    const void* h;
    const void* W;
    float* u;
    int P, d, R;
    float* ws = nullptr;  // optional split-K workspace (project_workspace_bytes)
    void* out_bf16 = nullptr;  // bf16 path only: write the output here in bf16 instead of u
};

struct EdgesArgs {
    const int32_t* cand_ids;
    const float* u;
    const void* A;
    const void* B;
    const float* unary;
    int S, n, K, R, V;
    float* edges_out;
    int32_t* best_slot;
    float* best_score;
    int32_t* err_flag;
};

struct ChainArgs {
    const int32_t* cand_ids;
    const float* unary;
    const float* edges;
    const int32_t* best_slot;
    const int32_t* start_slot;
    int S, n, K;
    float p_min;
    int32_t* tokens;
    float* probs;
    int32_t* length;
    int32_t* err_flag;
};

// Largest K the top-K kernel takes.
constexpr int kTopkMaxK = 1024;

struct TopkLaunch {
    const void* logits;
    int rows, V, K;
    int bf16;
    int32_t* ids;
    float* vals;
};

// 2-D bf16 tensor map over a row-major [rows, cols] array with a box of
// box_rows x 64 columns and 128-byte swizzle (out-of-range elements read as 0).
bool make_tmap_rows_bf16(CUtensorMap* m, const void* base, int rows, int cols, int box_rows);

// Each launcher enqueues on `stream` and returns the launch's cudaError_t.
cudaError_t launch_dynconv(const DynconvArgs& a, cudaStream_t stream);
// Reads and clears the convolution kernels' device fault word (synchronous).
cudaError_t take_dynconv_faults(unsigned* flags);

// The conv with its taps predicted from its input, fused (dynconv_pred.cu).
constexpr int kMaxPredT = 8;
struct DynconvPredArgs {
    const void* x;     // [S*n, C] bf16
    const void* hist;  // [S, T-1, C] bf16 or nullptr
    const void* base;  // [T, C] bf16
    const void* Wc;    // [T*G, C] bf16
    void* out;         // [S*n, C] bf16 or fp32
    int S, n, C, T, G;
    int out_bf16;
};
struct DynconvPredPlan {
    int NP, kblocks, m_tiles, split, stages, cdepth;
    uint32_t stage_bytes, ring_bytes, ds_bytes, tmem_cols;
    size_t smem_bytes;
};
// False when the shapes are outside what the fused kernel supports.
bool plan_dynconv_pred(const DynconvPredArgs& a, int num_sms, size_t max_smem, DynconvPredPlan* plan);
cudaError_t launch_dynconv_pred(const DynconvPredArgs& a, const DynconvPredPlan& plan,
                                cudaStream_t stream);
// fp32 inputs and output (T*G <= 256): delta in exact fp32, no tensor cores.
cudaError_t launch_dynconv_pred_f32(const DynconvPredArgs& a, cudaStream_t stream);
cudaError_t take_fused_faults(unsigned* flags);
cudaError_t launch_project_bf16_tc(const ProjectArgs& a, cudaStream_t stream, int num_sms);
// Bytes of split-K workspace the bf16 projection uses for these shapes (0: none).
size_t project_workspace_bytes(int P, int d, int R, int num_sms);
// Size of the library's own fixed projection workspace (8 MiB).
constexpr size_t kFixedProjectWorkspaceBytes = size_t(8) << 20;
// Device address of that workspace in the current context (looked up on every call).
cudaError_t fixed_project_workspace(float** ptr);
cudaError_t launch_project_f32(const ProjectArgs& a, cudaStream_t stream);
// Reads and clears the projection kernel's device fault word (synchronous).
cudaError_t take_project_faults(unsigned* flags);
// Tensor-core tile path: bf16 codebooks, K a power of two <= 128, R <= 384.
bool edges_tc_supported(int K, int R);
// u_only_dependency: the preceding kernel in the stream only produces u (and
// has itself waited for everything before it), so the kernel may read ids,
// codebooks and unary before that kernel completes.
cudaError_t launch_edges_bf16_tc(const EdgesArgs& a, int u_only_dependency, cudaStream_t stream);
// Warp-per-predecessor path (any K <= 256, R <= 512; fp32 or bf16 codebooks).
cudaError_t launch_edges_warp(const EdgesArgs& a, int cb_bf16, cudaStream_t stream);

// Greedy chain readout (one CTA per sequence; shared memory per CTA below).
size_t chain_smem_bytes(int n, int K);
cudaError_t launch_chain(const ChainArgs& a, cudaStream_t stream);

// Top-K candidate extraction (1 <= K <= min(V, kTopkMaxK)).
cudaError_t launch_topk(const TopkLaunch& a, cudaStream_t stream);
// Reads and clears the top-K kernel's device fault word (synchronous).
cudaError_t take_topk_faults(unsigned* flags);

// The composite selector in one kernel (select.cu): bf16, K a power of two in
// [4, 128], R in {64, 128, 256}, d % 8 == 0, n >= 2.
struct SelectArgs {
    const void* h;
    const void* W;
    const int32_t* cand_ids;
    const void* A;
    const void* B;
    const float* unary;
    int S, n, d, K, R, V;
    float* u;
    float* edges_out;
    int32_t* best_slot;
    float* best_score;
    int32_t* err_flag;
};
bool select_fused_supported(int K, int R, int d, int n);
// Sets *launched = false (and launches nothing) when no cluster layout fits the
// shapes; the caller then runs the projection and the edge kernel separately.
cudaError_t launch_select_fused(const SelectArgs& a, cudaStream_t stream, int num_sms,
                                size_t max_smem, bool* launched);
// The edge scores and argmax alone with the one-kernel selector's edge phase (u
// given; the same shapes as launch_select_fused with any d).  Sets *launched =
// false when the shapes are not covered; the caller then runs an edge kernel.
cudaError_t launch_select_edges(const EdgesArgs& a, cudaStream_t stream, int num_sms,
                                size_t max_smem, bool* launched);
// Whether launch_select_fused runs for these shapes, and its cluster layout.
bool select_fused_plan(int S, int n, int d, int K, int R, int num_sms, size_t max_smem,
                       int* cluster_size, int* clusters, int* rows_per_block);
// Reads and clears the fused selector's device fault word (synchronous).
cudaError_t take_select_faults(unsigned* flags);

// Distillation from a teacher's top-K logits (distill.cu).  loss and lse, with
// grad when it is not nullptr; or, when grad_loss is not nullptr, the gradient
// alone from it and lse.
struct DistillArgs {
    const void* logits;    // [rows, V], rows `ld` elements apart
    long long ld;
    const int32_t* ids;    // [rows, K]
    const float* teacher;  // [rows, K]
    const float* weight;   // [rows] or nullptr (1)
    const float* grad_loss;  // [rows] or nullptr
    int rows, V, K;
    float inv_t, c;        // 1 / T and log2(e) / T
    float* loss;
    float* lse;
    void* grad;            // [rows, V], rows `grad_ld` elements apart
    long long grad_ld;
    int32_t* err_flag;
    int lg = 0, per = 0, ring = 0;  // the split of a row, set by the launcher
};
constexpr int kDistillMaxK = 1024;
constexpr int kDistillMaxV = 1 << 28;
cudaError_t launch_distill(DistillArgs a, int bf16, cudaStream_t stream, int num_sms);

// One token of every row by temperature, top-k, top-p and min-p (sample.cu).  A
// setting's pointer, when not nullptr, has a value for every row.
struct SampleArgs {
    const void* logits;  // [rows, V], rows `ld` elements apart
    long long ld;
    const float* uniform;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    float temperature0;
    int top_k0;
    float top_p0, min_p0;
    int rows, V;
    int32_t* tokens;
    float* probs;        // [rows] or nullptr
    int lg = 0, per = 0, ring = 0;  // the split of a row, set by the launcher
};
// Largest V: the fixed-point sums of a row stay inside 62 bits, and those of a
// CTA's histogram inside their words.
constexpr int kSampleMaxV = 1 << 21;
cudaError_t launch_sample(SampleArgs a, int bf16, cudaStream_t stream, int num_sms);

// Losses of a token's log-probability by row (token_loss.cu): the clipped policy loss with a
// KL term, and the preference loss of pairs of sequences.
struct TokenLossArgs {
    const void* logits;   // [rows, V], rows `ld` elements apart
    long long ld;
    const int32_t* tokens;  // [rows], negative: none
    int rows, V;
    float inv_t, c;       // 1 / T and log2(e) / T
    const float* weight;  // [rows] (policy) or [pairs], or nullptr (1)
    const float* ref_logp;  // [rows], or [2 * pairs] or nullptr
    const float* grad_loss;  // [rows] or [pairs]; nullptr in the call with the loss
    // policy
    const float* old_logp;  // [rows]
    const float* advantage;  // [rows]
    float ratio_lo, ratio_hi, kl_coef;
    // preference: sequence s has the rows offsets[s] to offsets[s + 1]; pair i consists of the
    // chosen one i and the rejected one pairs + i
    const int32_t* offsets;  // [2 * pairs + 1]
    int pairs, average;
    float beta, smoothing, margin;
    float* seq_logp;      // [2 * pairs]
    float* loss;          // [rows] or [pairs]
    float* logp;          // [rows]
    float* lse;           // [rows]
    void* grad;           // [rows, V], rows `grad_ld` elements apart, or nullptr
    long long grad_ld;
    int32_t* err_flag;
    int keep = 0;         // the last rows, which a pass that follows should find in L2
    int lg = 0, per = 0, ring = 0;  // the split of a row, set by the launcher
};
enum class TokenLossPass { kLoss, kGrad };  // the loss (with grad when it is set); grad alone
cudaError_t launch_policy_loss(const TokenLossArgs& a, TokenLossPass pass, int bf16,
                               cudaStream_t stream, int num_sms);
cudaError_t launch_preference_loss(const TokenLossArgs& a, TokenLossPass pass, int bf16,
                                   cudaStream_t stream, int num_sms);

// Steps on the weights of many tensors (adamw.cu).  The arrays have an entry for each tensor and
// are read during the call.
struct GradNormArgs {
    int count;
    const void* const* grads;
    const long long* sizes;
    double* workspace;   // grad_norm_chunks(...) values
    float* norm;
};
// Values of workspace: one for each chunk, none where a single launch does.
long long grad_norm_chunks(int count, const long long* sizes);
cudaError_t launch_grad_norm(const GradNormArgs& a, int grad_bf16, cudaStream_t stream);

struct AdamwArgs {
    int count;
    void* const* params;
    const void* const* grads;
    void* const* exp_avg;
    void* const* exp_avg_sq;
    float* const* master;             // or nullptr
    uint8_t* const* exp_avg_scale;    // 8-bit states, or nullptr
    uint8_t* const* exp_avg_sq_scale;
    const long long* sizes;
    const int32_t* step_at;           // on the device, or nullptr: `step`
    const float* lr_at;               // on the device, or nullptr: `lr`
    int step;
    double lr, beta1, beta2, eps, weight_decay;
    const float* norm;                // on the device, or nullptr
    double max_norm;                  // 0: no limit
    double grad_scale;
    int by_chance;
    unsigned long long seed;
};
cudaError_t launch_adamw(const AdamwArgs& a, int param_bf16, int grad_bf16, cudaStream_t stream);

// 8-bit optimizer states to values and back (to the nearest).
cudaError_t launch_state_decode(const uint8_t* codes, const uint8_t* scale, long long n, int squares,
                                void* out, int out_bf16, cudaStream_t stream);
cudaError_t launch_state_encode(const void* values, int in_bf16, long long n, int squares,
                                uint8_t* codes, uint8_t* scale, cudaStream_t stream);

// Measurement aid: random-row gather (probe.cu).  out[i] = XOR of the 32-bit
// words of row ids[i] (ids clamped into [0, rows)); row_bytes a power of two
// in [16, 512].
struct ProbeGatherArgs {
    const void* table;
    long long rows;
    int row_bytes;
    const int32_t* ids;
    int n_ids;
    uint32_t* out;
};
cudaError_t launch_probe_gather(const ProbeGatherArgs& a, cudaStream_t stream, int num_sms);

}  // namespace df2
