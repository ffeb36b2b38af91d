"""Layers of an FP8 checkpoint's feed-forward half, as a program would run them, for one token or thousands.

The library's calls in the order of a layer: residual add and norm to 8-bit activations (residual_norm), both
projections with SiLU(gate) * up, h written as the down projection's 8-bit input (fp8_b128_gemm_silu_mul), and the down
projection (fp8_b128_gemm), whose rows the next layer's residual_norm adds; before the first layer an output projection
of rows that no norm precedes (fp8_x_encode, fp8_b128_gemm). PyTorch holds the memory and makes random weights in the
checkpoint's form: E4M3 codes and one fp32 scale for each 128 x 128 tile.

    python examples/fp8_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_decode_nvfp4_gb300 as bqd  # noqa: E402


def blocks(n):
    return -(-n // 128)


class Weight:
    """FP8 block-128 weights [M][K] of a random matrix, codes and tile scales."""

    def __init__(self, M, K, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.zeros(blocks(M) * 128, blocks(K) * 128, device="cuda")
        w[:M, :K] = torch.randn(M, K, generator=g, device="cuda") / math.sqrt(K)
        tiles = w.view(blocks(M), 128, blocks(K), 128)
        self.M, self.K = M, K
        self.scales = (tiles.abs().amax((1, 3)) / 448.0).contiguous()
        self.codes = (tiles / self.scales[:, None, :, None]).view(w.shape)[:M, :K].to(torch.float8_e4m3fn).contiguous()

    def values(self):
        s = self.scales.double().repeat_interleave(128, 0)[:self.M].repeat_interleave(128, 1)[:, :self.K]
        return self.codes.double() * s


class Activations:
    """8-bit activations of up to `tokens` tokens of K channels; buffers that a program keeps from step to step."""

    def __init__(self, tokens, K):
        self.K = K
        self.codes = torch.empty(tokens * K, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(blocks(K) * tokens, device="cuda")

    def values(self, T):
        s = self.scales[:blocks(self.K) * T].view(-1, T).double().t().repeat_interleave(128, 1)[:, :self.K]
        return self.codes[:T * self.K].view(T, self.K).view(torch.float8_e4m3fn).double() * s


class Model:
    def __init__(self, hidden=512, inner=1152, layers=2, tokens=512, eps=1e-6, seed=0):
        self.hidden, self.inner, self.eps = hidden, inner, eps
        self.out = Weight(hidden, hidden, seed)
        self.layers = [dict(gate=Weight(inner, hidden, seed + 3 * i + 1), up=Weight(inner, hidden, seed + 3 * i + 2),
                            down=Weight(hidden, inner, seed + 3 * i + 3), norm=torch.ones(hidden, device="cuda"))
                       for i in range(layers)]
        self.final = torch.ones(hidden, device="cuda")
        self.x, self.h = Activations(tokens, hidden), Activations(tokens, inner)
        self.rows = torch.empty(tokens, hidden, device="cuda")

    def step(self, attention, residual):
        """bf16 rows [T][hidden] of attention, fp32 residual [T][hidden] (updated): the last norm's bf16 rows."""
        T, H, x, h = attention.shape[0], self.hidden, self.x, self.h
        rows = self.rows[:T]
        bqd.fp8_x_encode(attention, bqd.BQD_BF16, H, x.codes, x.scales, H, T)
        bqd.fp8_b128_gemm(self.out.codes, self.out.scales, x.codes, x.scales, rows, bqd.BQD_F32, H, H, T)
        for layer in self.layers:
            gate, up, down = layer["gate"], layer["up"], layer["down"]
            bqd.residual_norm(rows, bqd.BQD_F32, H, None, None, 0, 0, 1.0, residual, residual, bqd.BQD_F32, layer["norm"],
                              self.eps, x.codes, bqd.BQD_E4M3, x.scales, H, T)
            bqd.fp8_b128_gemm_silu_mul(gate.codes, gate.scales, up.codes, up.scales, x.codes, x.scales, h.codes,
                                       bqd.BQD_E4M3, h.scales, self.inner, H, T)
            bqd.fp8_b128_gemm(down.codes, down.scales, h.codes, h.scales, rows, bqd.BQD_F32, H, self.inner, T)
        y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        bqd.residual_norm(rows, bqd.BQD_F32, H, None, None, 0, 0, 1.0, residual, residual, bqd.BQD_F32, self.final, self.eps,
                          y, bqd.BQD_BF16, None, H, T)
        return y


def main():
    model = Model()
    for T in (1, 40, 300):
        attention = torch.randn(T, model.hidden, device="cuda").to(torch.bfloat16)
        y = model.step(attention, torch.randn(T, model.hidden, device="cuda"))
        print(f"{T} tokens: {tuple(y.shape)}, mean square {float((y.float() ** 2).mean()):.3f}")


if __name__ == "__main__":
    main()
