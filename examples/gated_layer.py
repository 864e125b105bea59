"""One layer's feed-forward half with a gate of its own, prefill and single-token decode.

    python examples/gated_layer.py [--tokens 512]

The attention output is projected and added to the residual stream (moe_linear), the router's fp32
logits come from another projection, a sigmoid gate with a balance bias picks 8 of 256 experts in 4 of 8
groups (moe_gate), the choice becomes the routing of the 4-bit experts (moe_dispatch), and the experts'
combined output closes the layer.  The last tokens go through a vocabulary head.  Weights and inputs are
synthetic; a sample of tokens is compared with the CPU oracle.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_grouped_gemm_gb300 as moe  # noqa: E402
from moe_workload import configs  # noqa: E402


def device(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


class GatedLayer:
    """The weights of a layer, and the configs, routing and workspaces for T tokens a call."""

    def __init__(self, T: int, d: int = 2048, I: int = 512, attention: int = 4096, vocab: int = 32768, seed: int = 1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(n, k):
            return torch.empty(n, k, device="cuda").normal_(0, k ** -0.5, generator=g).bfloat16()

        wl = configs.custom_workload("gated_layer", T=T, d=d, I=I)
        self.inputs = configs.make_layer(wl)
        self.shape = moe.shape(T, d, 256, 8, I, I)
        pack = lambda m: (device(m.codes), device(m.scales), device(m.biases))  # noqa: E731
        r, s = self.inputs.routed, self.inputs.shared
        self.routed = moe.moe_pack_weights(self.shape, pack(r.gate), pack(r.up), pack(r.down), I)
        self.shared = moe.moe_pack_weights(self.shape, pack(s.gate), pack(s.up), pack(s.down), I)
        self.w_out, self.w_router, self.w_head = matrix(d, attention), matrix(256, d), matrix(vocab, d)
        self.balance = 0.05 * torch.randn(256, device="cuda", generator=g)

        self.out = moe.linear_config(T, d, attention)                                   # + residual
        self.router = moe.linear_config(T, 256, d, out_dtype=torch.float32)
        self.gate = moe.gate_config(T, 256, 8, score="sigmoid", groups=8, group_topk=4, scale=2.5)
        self.head = moe.linear_config(min(T, 16), vocab, d, out_dtype=torch.float32)
        self.ws = [moe.linear_workspace(c) for c in (self.out, self.router, self.head)]
        self.moe_ws = moe.workspace(self.shape)
        self.routing = moe.Routing(T)
        self.hidden = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty(T, 256, device="cuda")
        self.y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        self.next = torch.empty(min(T, 16), vocab, device="cuda")

    def __call__(self, attention: torch.Tensor, residual: torch.Tensor):
        """attention [T, attention], residual [T, d] (bf16) -> experts' output [T, d], logits of the last tokens."""
        moe.moe_linear(self.out, attention, self.w_out, None, residual, self.hidden, self.ws[0])
        moe.moe_linear(self.router, self.hidden, self.w_router, None, None, self.logits, self.ws[1])
        moe.moe_gate(self.gate, self.logits, self.balance, self.routing.topk_idx, self.routing.topk_w)
        moe.moe_dispatch(self.shape, self.hidden, self.routing, self.moe_ws)
        moe.moe_grouped_ffn(self.shape, self.hidden, self.routing, self.routed, self.shared, self.moe_ws)
        moe.moe_combine(self.shape, self.routing, self.moe_ws, self.y)
        n = self.next.shape[0]
        moe.moe_linear(self.head, self.y[-n:], self.w_head, None, None, self.next, self.ws[2])
        return self.y, self.next

    def check_status(self) -> None:
        for ws in self.ws + [self.moe_ws]:
            rc, bits = moe.moe_read_status(ws)
            if rc != moe.MOE_OK:
                raise RuntimeError(f"device status {bits:#x}")


def compare_with_oracle(layer: GatedLayer, tokens) -> float:
    """Relative Frobenius error of the experts' output for some tokens, given the layer's own hidden state and choice."""
    import oracle
    oracle.build()
    x = layer.hidden.view(torch.int16).cpu().numpy().view(np.uint16)
    idx, w = layer.routing.topk_idx.cpu().numpy(), layer.routing.topk_w.cpu().numpy().astype(np.float64)
    ref = oracle.moe_tokens(x, idx, w, layer.inputs.routed, layer.inputs.shared, tokens)
    got = layer.y[torch.as_tensor(np.asarray(tokens)).cuda()].double().cpu().numpy()
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    args = ap.parse_args()
    for T in (args.tokens, 1):
        layer = GatedLayer(T)
        attention = torch.randn(T, 4096, device="cuda").bfloat16()
        residual = torch.randn(T, 2048, device="cuda").bfloat16()
        for _ in range(3):
            layer(attention, residual)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            y, logits = layer(attention, residual)
        end.record()
        end.synchronize()
        layer.check_status()
        err = compare_with_oracle(layer, sorted({0, T // 2, T - 1}))
        print(f"{T} token(s): {start.elapsed_time(end) / 20 * 1e3:.1f} us a pass; next tokens "
              f"{logits.argmax(1)[-4:].tolist()}; experts against the oracle {err:.1e}")


if __name__ == "__main__":
    main()
