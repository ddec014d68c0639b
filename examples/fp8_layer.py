"""A layer of an FP8 sampler on the view that the receiver keeps, on one GPU.

The trainer changes a few of the weights and sends their patch.  The receiver applies it to its BF16
view and quantises the view in the same pass.  Then a layer runs on the codes: norm, [gate; up],
the activation, down; behind it an expert layer for a few tokens; and, for adapters trained
over the frozen codes, the gradient of the layer's input.

    python -m examples.fp8_layer [tokens]
"""
import sys

import torch

import sparse_delta_codec_amd as pulse

HIDDEN, INTER, EXPERTS, EXPERT_INTER, TOP_K = 512, 768, 6, 256, 2
EPS = 1e-6


def _normal(shape, std, gen):
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen).to(torch.bfloat16)


def _blocks(n):
    return -(-n // 128)


def _codes(*shape):
    """Codes of a matrix and its scales for each 128 x 128 block."""
    return (torch.zeros(shape, dtype=torch.uint8, device="cuda"),
            torch.zeros(*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]), device="cuda"))


def _rows(t, cols):
    """Codes of rows and their scales for each 128 columns."""
    return torch.zeros(t, cols, dtype=torch.uint8, device="cuda"), torch.zeros(t, _blocks(cols), device="cuda")


class View:
    """What the receiver keeps: the weights as one BF16 view, and their codes."""

    def __init__(self, gen):
        self.sizes = [HIDDEN, INTER * HIDDEN, INTER * HIDDEN, HIDDEN * INTER, HIDDEN]
        at = [sum(self.sizes[:i]) for i in range(6)]
        self.bf16 = torch.cat([1 + _normal(HIDDEN, 0.1, gen), _normal(2 * INTER * HIDDEN, HIDDEN ** -0.5, gen),
                               _normal(HIDDEN * INTER, INTER ** -0.5, gen), 1 + _normal(HIDDEN, 0.1, gen)])
        self.norm, self.last_norm = self.bf16[:HIDDEN], self.bf16[at[4]:]
        self.up, self.up_scales = _codes(2 * INTER, HIDDEN)
        self.down, self.down_scales = _codes(HIDDEN, INTER)
        n = at[5]
        self.plan = pulse.pulse_apply_quant_plan(
            [([(at[0], 1)], HIDDEN, None, None), ([(at[1], INTER), (at[2], INTER)], HIDDEN, self.up.view(-1), self.up_scales.view(-1)),
             ([(at[3], HIDDEN)], INTER, self.down.view(-1), self.down_scales.view(-1)), ([(at[4], 1)], HIDDEN, None, None)], n)
        self.ws = pulse.workspace(pulse.PULSE_OP_APPLY_QUANT, n, 0)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # the experts come whole, all of a kind in one call
        gate, up = _normal((EXPERTS, EXPERT_INTER, HIDDEN), HIDDEN ** -0.5, gen), _normal((EXPERTS, EXPERT_INTER, HIDDEN), HIDDEN ** -0.5, gen)
        self.experts_up, self.experts_up_scales = _codes(EXPERTS, 2 * EXPERT_INTER, HIDDEN)
        self.experts_down, self.experts_down_scales = _codes(EXPERTS, HIDDEN, EXPERT_INTER)
        down = _normal((EXPERTS, HIDDEN, EXPERT_INTER), EXPERT_INTER ** -0.5, gen)
        pulse.fp8_block_quant([gate, up], self.experts_up, self.experts_up_scales, batch=EXPERTS)
        pulse.fp8_block_quant([down], self.experts_down, self.experts_down_scales, batch=EXPERTS)
        self.router = _normal((EXPERTS, HIDDEN), 1.0, gen).float()

    def update(self, idx, val, count):
        """The patch applied, and the codes of the new weights."""
        pulse.pulse_apply_quant(self.bf16, idx, val, count, self.plan, self.status, self.ws)


class Layer:
    """The buffers of a layer for `t` tokens, and its passes."""

    def __init__(self, view, t):
        self.view, self.t = view, t
        bf16 = lambda cols: torch.zeros(t, cols, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.x_scales = _rows(t, HIDDEN)
        self.h, self.h_scales = _rows(t, INTER)
        self.rstd = torch.zeros(t, device="cuda")
        self.both, self.out, self.last, self.mixed = bf16(2 * INTER), bf16(HIDDEN), bf16(HIDDEN), bf16(HIDDEN)
        self.logits = torch.zeros(t, EXPERTS, device="cuda")
        self.ids = torch.zeros(t, TOP_K, dtype=torch.int32, device="cuda")
        self.shares = torch.zeros(t, TOP_K, device="cuda")
        self.ws = [pulse.fp8_gemm_workspace(t, 2 * INTER, HIDDEN), pulse.fp8_gemm_workspace(t, HIDDEN, INTER),
                   pulse.moe_workspace(t, HIDDEN, EXPERT_INTER, EXPERTS, TOP_K)]
        # for the gradients
        self.dy, self.dy_scales = _rows(t, HIDDEN)
        self.dboth, self.dboth_scales = _rows(t, 2 * INTER)
        self.dh, self.dnorm, self.dx = bf16(INTER), bf16(HIDDEN), bf16(HIDDEN)
        self.dweight = torch.zeros(HIDDEN, device="cuda")
        self.back_ws = [pulse.fp8_gemm_workspace(t, HIDDEN, INTER, form="nn"),
                        pulse.fp8_gemm_workspace(t, 2 * INTER, HIDDEN, form="nn"), pulse.rms_norm_workspace(t, HIDDEN)]

    def forward(self, x, stream):
        """The layer's output in self.mixed; `stream`, the residual stream, has x and the MLP added."""
        v = self.view
        pulse.pulse_rms_norm(x, v.norm, EPS, residual=stream, codes=self.x, scales=self.x_scales, rstd=self.rstd)
        pulse.fp8_block_gemm(self.x, self.x_scales, v.up, v.up_scales, self.both, self.ws[0])
        pulse.fp8_group_quant(self.both, self.h, self.h_scales, glu=True)
        pulse.fp8_block_gemm(self.h, self.h_scales, v.down, v.down_scales, self.out, self.ws[1])
        pulse.pulse_rms_norm(self.out, v.last_norm, EPS, residual=stream, y=self.last)
        torch.mm(self.last.float(), v.router.t(), out=self.logits)
        pulse.pulse_moe_route(self.logits, self.ids, self.shares)
        pulse.pulse_moe_forward(self.last, self.ids, self.shares, v.experts_up, v.experts_up_scales, v.experts_down,
                                v.experts_down_scales, self.mixed, v.status, self.ws[2])
        return self.mixed

    def backward(self, before, dy):
        """dx of the MLP's input and its norm's dweight, for a gradient dy of the stream behind the MLP;
        `before`: the stream in front of it, as the norm left it."""
        v = self.view
        pulse.fp8_group_quant(dy, self.dy, self.dy_scales)
        pulse.fp8_block_gemm(self.dy, self.dy_scales, v.down, v.down_scales, self.dh, self.back_ws[0], form="nn")
        gate, up = self.both.float().chunk(2, dim=1)
        s, d = torch.sigmoid(gate), self.dh.float()
        self.dgate_up = torch.cat([d * up * s * (1 + gate * (1 - s)), d * gate * s], dim=1).to(torch.bfloat16)
        pulse.fp8_group_quant(self.dgate_up, self.dboth, self.dboth_scales)
        pulse.fp8_block_gemm(self.dboth, self.dboth_scales, v.up, v.up_scales, self.dnorm, self.back_ws[1], form="nn")
        pulse.pulse_rms_norm_backward(before, v.norm, self.rstd, self.dnorm, self.dx, self.dweight, self.back_ws[2], dres=dy)
        return self.dx


def patch(gen, n, share=0.01):
    """A patch of `share` of the view's elements, as a trainer's step leaves it."""
    idx = torch.randperm(n, generator=gen, device="cuda")[:max(1, int(n * share))].sort().values.to(torch.int32)
    val = _normal(idx.numel(), 0.05, gen)
    return idx, val, torch.tensor([idx.numel()], dtype=torch.int64, device="cuda")


def run(tokens=20, seed=0):
    """(view, layer, x, the stream in front, behind the norm and at the end, dy)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    view = View(gen)
    view.update(*patch(gen, view.bf16.numel()))
    layer = Layer(view, tokens)
    x, stream, dy = _normal((tokens, HIDDEN), 0.5, gen), _normal((tokens, HIDDEN), 1.0, gen), _normal((tokens, HIDDEN), 1e-2, gen)
    front = stream.clone()
    layer.forward(x, stream)
    before = (x.float() + front.float()).to(torch.bfloat16)
    layer.backward(before, dy)
    torch.cuda.synchronize()
    return view, layer, x, front, before, stream, dy


if __name__ == "__main__":
    view, layer, *_ = run(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
    assert int(view.status.item()) == 0
    print(f"{layer.t} tokens: |y| {layer.mixed.float().norm():.3f}, |dx| {layer.dx.float().norm():.4f}, experts "
          f"{torch.bincount(layer.ids.flatten(), minlength=EXPERTS).tolist()}")
