// fp8.h -- internal launchers of the calls on 8-bit activations: their
// encoder and the norm that writes them (fp8_rows.cu), and the products with
// FP8 block-128 weights (fp8_gemm.cu). Arguments are checked by the callers
// (abi.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bqd.h"

namespace bqd {

struct EncodeXArgs {
    const void* x;
    int64_t pitch;
    uint8_t* codes;
    float* scales;
    int64_t K, T;
};
cudaError_t launch_fp8_x_encode(const EncodeXArgs& a, int x_type, cudaStream_t s);

constexpr int64_t kNormMaxH = 16384;

struct NormArgs {
    const void *x, *gate, *residual;
    void *residual_out, *y;
    const float *post_weight, *pre_weight;
    float* y_scales;
    int64_t x_pitch, gate_pitch, T;
    float scale, eps;
    int H, x_f32, gate_f32, res_f32, y_e4m3;
};
cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t s);

struct Fp8GemmArgs {
    const uint8_t *w0, *w1;  // weights [M][K]; w1: the up projection (dual form), else unused
    const float *s0, *s1;    // their tile scales [ceil(M/128)][ceil(K/128)]
    const uint8_t* x;        // [T][K]
    const float* xs;         // [ceil(K/128)][T]
    void* y;                 // [T][M]
    float* ys;               // [ceil(M/128)][T] with E4M3 outputs
    int64_t M, K, T;
    int y_type;
};
// Codes [rows][K] in boxes of 128 k x `box` rows (a CUtensorMap); k and rows past the ends read as zero.
bool fp8_codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box);
// fp32 or bf16 outputs [rows][M], whole 16 bytes a row, in boxes of `line` (128) bytes x `box` rows.
bool fp8_rows_map(CUtensorMap* map, void* y, int y_type, int64_t rows, int64_t M, int box, int line);
// The kernel for more than 64 tokens (fp8_gemm_tokens.cu).
cudaError_t launch_fp8_gemm_tokens(const Fp8GemmArgs& a, bool dual, cudaStream_t s);
// The kernel for many tokens (fp8_gemm_pairs.cu), and whether the sizes are its.
bool fp8_gemm_wants_pairs(const Fp8GemmArgs& a, bool dual);
cudaError_t launch_fp8_gemm_pairs(const Fp8GemmArgs& a, bool dual, cudaStream_t s);
bool fp8_gemm_supported(int64_t M, int64_t K, int64_t T);
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, bool dual, cudaStream_t s);
cudaError_t read_and_clear_fp8_error(unsigned int* out);
cudaError_t read_and_clear_fp8_pairs_error(unsigned int* out);
cudaError_t read_and_clear_fp8_tokens_error(unsigned int* out);

}  // namespace bqd
