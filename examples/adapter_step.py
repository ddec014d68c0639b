"""RL post-training of low-rank adapters, trainer to sampler, on one GPU.

A frozen projection y = x W^T carries one low-rank adapter per task.  The trainer
runs a batch of several tasks through the projection and its adapters, forward and
backward; clips the gradients by their norm; takes an AdamW step on the float32
masters with 8-bit states, which writes the BF16 adapters that the projection reads
and the sparse patch of their changed elements.  The sampler applies the patch to
its own copy and serves one token of each of many requests with it: bit for bit what
the trainer's adapters give.

    python -m examples.adapter_step [steps]
"""
import sys

import torch

import sparse_delta_codec_amd as pulse

K, N, RANK, TASKS = 1024, 768, 16, 6
PROMPTS = 24            # prompts of a training batch, of 16 to 100 tokens
REQUESTS = 64           # requests the sampler serves a token of


def _normal(shape, std, gen, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


class Adapters:
    """BF16 adapter pools, as the projection reads them."""

    def __init__(self, a, b):
        self.a, self.b = a, b
        self.scales = torch.full((TASKS,), 2.0, device="cuda")

    def apply(self, x, ids, y, plan, ws, status, h=None):
        pulse.pulse_lora_plan(plan, ids, status)
        pulse.pulse_lora_forward(x, self.a, self.b, self.scales, plan, y, ws, h=h)


class Trainer:
    def __init__(self, gen, max_tokens):
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # A starts random and B at zero, so that the adapters start as nothing
        self.masters = [_normal((TASKS, RANK, K), K ** -0.5, gen, torch.float32),
                        torch.zeros(TASKS, RANK, N, device="cuda")]
        self.views = [p.to(torch.bfloat16) for p in self.masters]
        self.adapters = Adapters(*self.views)
        self.grads = [torch.zeros_like(p) for p in self.masters]
        codes = [[torch.zeros(p.numel(), dtype=torch.uint8, device="cuda") for p in self.masters] for _ in "mv"]
        scales = [[torch.zeros(-(-p.numel() // pulse.PULSE_ADAMW_BLOCK), device="cuda") for p in self.masters] for _ in "mv"]
        self.table = pulse.AdamWTable(self.masters, self.grads, *codes, b=self.views, m_scale=scales[0], v_scale=scales[1],
                                      weight_decay=0.01)
        self.norms = pulse.GradTable(self.grads)
        self.clip = torch.zeros(2, device="cuda")  # the factor on the gradients, and their norm
        self.norm_ws = pulse.workspace(pulse.PULSE_OP_GRAD_NORM, self.norms.ntiles)
        self.step_ws = pulse.workspace(pulse.PULSE_OP_ADAMW, self.table.ntiles)
        total = sum(p.numel() for p in self.masters)
        self.patch_idx = torch.zeros(total, dtype=torch.int32, device="cuda")
        self.patch_val = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
        self.patch_offsets = torch.zeros(len(self.masters) + 1, dtype=torch.int64, device="cuda")
        self.plan = pulse.LoraPlan(max_tokens, TASKS)
        self.ws = pulse.lora_workspace(max_tokens, K, N, RANK, TASKS, train=True)
        self.h = pulse.lora_hidden(max_tokens, RANK, TASKS)
        self.steps = 0

    def step(self, weight, x, ids, target, lr=1e-3):
        """One training step; returns the loss.  The patch is left in patch_*."""
        y = x @ weight.t()
        self.adapters.apply(x, ids, y, self.plan, self.ws, self.status, h=self.h)
        error = y.float() - target
        dy = (error * (2.0 / error.numel())).to(torch.bfloat16)
        # the frozen projection's own input gradient would go into dx first; nothing below needs it here
        pulse.pulse_lora_backward(x, dy, self.views[0], self.views[1], self.adapters.scales, self.plan, self.h, None,
                                  *self.grads, self.ws)
        self.steps += 1
        pulse.pulse_grad_norm(self.norms, self.clip, self.norm_ws, max_norm=1.0)
        pulse.pulse_adamw_step(self.table, self.steps, lr, d_scale=self.clip, seed=self.steps, d_status=self.status,
                               ws=self.step_ws, patch_idx=self.patch_idx, patch_val=self.patch_val,
                               seg_offsets=self.patch_offsets)
        return error.square().mean()


class Sampler:
    def __init__(self, trainer):
        self.views = [v.clone() for v in trainer.views]
        self.adapters = Adapters(*self.views)
        self.table = pulse.ViewTable(self.views)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.plan = pulse.LoraPlan(REQUESTS, TASKS)
        self.ws = pulse.lora_workspace(REQUESTS, K, N, RANK, TASKS)

    def receive(self, trainer):
        pulse.pulse_apply_patch_segments(self.table, trainer.patch_idx, trainer.patch_val, trainer.patch_offsets,
                                         self.status)

    def decode(self, weight, x, ids):
        y = x @ weight.t()
        self.adapters.apply(x, ids, y, self.plan, self.ws, self.status)
        return y


def run(steps=20, seed=0):
    """Trains and serves; returns the losses, the shares of the adapters that the patches
    carried, and whether the sampler's tokens equal the trainer's in every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    weight = _normal((N, K), K ** -0.5, gen)
    lengths = torch.randint(16, 101, (PROMPTS,), generator=host)
    tasks = torch.randint(-1, TASKS, (PROMPTS,), generator=host)  # -1: the projection as it is
    ids = torch.repeat_interleave(tasks, lengths).to(torch.int32).cuda()
    x = _normal((ids.numel(), K), 1.0, gen)
    target = (x.float() @ weight.float().t()) + (ids >= 0).float()[:, None]  # every task: its outputs one higher
    trainer = Trainer(gen, ids.numel())
    sampler = Sampler(trainer)
    request_ids = torch.randint(-1, TASKS, (REQUESTS,), generator=host).to(torch.int32).cuda()
    tokens = _normal((REQUESTS, K), 1.0, gen)
    total, losses, shares, same = sum(p.numel() for p in trainer.masters), [], [], True
    for _ in range(steps):
        losses.append(float(trainer.step(weight, x, ids, target)))
        sampler.receive(trainer)
        served, wanted = sampler.decode(weight, tokens, request_ids), tokens @ weight.t()
        trainer.adapters.apply(tokens, request_ids, wanted, sampler.plan, sampler.ws, trainer.status)
        same = same and torch.equal(served, wanted)
        shares.append(int(trainer.patch_offsets[-1]) / total)
    same = same and all(torch.equal(p, q) for p, q in zip(trainer.views, sampler.views))
    assert int(trainer.status) == 0 and int(sampler.status) == 0
    return losses, shares, same


if __name__ == "__main__":
    losses, shares, same = run(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
    for i, (loss, share) in enumerate(zip(losses, shares)):
        print(f"step {i + 1:3d}  loss {loss:.4f}  patch {share:.1%} of the adapters")
    print("the sampler's tokens equal the trainer's:", same)
