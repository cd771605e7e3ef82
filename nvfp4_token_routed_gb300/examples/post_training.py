"""Post-training of a small routed model whose experts stay frozen in NVFP4.

    python -m nvfp4_token_routed_gb300.examples.post_training

The model: tokens x [T, H]; a router (plain top-K) and the NVFP4 expert layer on
them, added to x; a head of V logits.  The router and the head learn, first by
distillation from a teacher's top logits (the same experts with BF16
activations, and the head before it was disturbed), then by the clipped policy
loss on sampled tokens, with the balance and z losses of the router all along.
Every forward, loss and gradient at the logits runs in the library; the dense
products of router and head are torch's.
"""
import torch

import nvfp4_token_routed_gb300 as M
from nvfp4_token_routed_gb300 import workloads as W

LAYER = W.Workload("post_training_T384_H256_I256_E16_K4", 384, 256, 256, 16, 4, "swiglu",
                   x_dist="normal")
VOCAB, TEACHER_TOP = 2000, 32
BALANCE, Z = 1e-2, 1e-3


class RoutedModel:
    def __init__(self, wl=LAYER, vocab=VOCAB, device="cuda", seed=7):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        w1, w2 = W.make_weights(wl, device=device, seed=seed)
        self.wl = wl
        self.experts = M.prepare_weights(w1, w2, wl.act)
        self.router = torch.randn(wl.E, wl.H, generator=g, device=device) * wl.H ** -0.5
        self.head = torch.randn(vocab, wl.H, generator=g, device=device) * (4.0 * wl.H ** -0.5)
        self.ws = M.workspace(self.experts, wl.T, wl.K, device=device)
        self.layout = M.moe_nvfp4_workspace_layout(self.experts.dims, wl.T, wl.K)

    def forward(self, x):
        """Logits [T, V] bf16, and what the backward pass needs."""
        r = x.float() @ self.router.t()
        ids, w = M.route_topk(r, self.wl.K)
        codes, sf, scale = M.quantize_tokens(x)
        h = x + M.forward(self.experts, codes, sf, scale, ids, w, ws=self.ws)
        return h @ self.head.to(torch.bfloat16).t(), (x, r, ids, w, h)

    def teacher_top(self, x, head, k=TEACHER_TOP):
        """Top logits of the same experts with BF16 activations and another head."""
        ids, w = M.route_topk(x.float() @ self.router.t(), self.wl.K)
        h = x + M.forward_w4a16(self.experts, x, ids, w)
        z = h.float() @ head.t()
        top = torch.topk(z, k, dim=1)
        return top.indices, top.values, torch.logsumexp(z, 1)

    def step(self, saved, dz, offsets, mask, rate):
        """One descent step of head and router; returns the router's losses and the load."""
        x, r, ids, w, h = saved
        dh = dz.float() @ self.head
        # the output is sum_k w_k y_k: each score's gradient is its expert row against dh
        rows = M.ws_view(self.ws, self.layout, "route", torch.bfloat16,
                         (self.layout["rows_cap"], M.padded(self.wl.H)))
        inv = M.ws_view(self.ws, self.layout, "inv", torch.int32, (self.wl.T, self.wl.K))
        y = rows[inv.long().clamp_min(0)][..., :self.wl.H].float()
        dw = (y * dh.unsqueeze(1)).sum(-1)
        losses, counts, tokens = M.router_loss(r, ids, BALANCE, Z, seq_offsets=offsets,
                                               token_mask=mask)
        dr = M.router_loss_grad(r, ids, counts, tokens, BALANCE, Z, seq_offsets=offsets,
                                token_mask=mask, topk_w=w, d_topk_w=dw, dlogits=r)
        self.head -= rate * (dz.float().t() @ h.float())
        self.router -= rate * (dr.t() @ x.float())
        return losses, counts


def run(distill_steps=20, policy_steps=12, device="cuda", seed=3):
    """Mean distillation loss and mean reward, step by step."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    wl = LAYER
    model = RoutedModel(wl, device=device)
    x = W.make_x(wl, device=device, seed=seed)
    # three packed sequences; the tail of the last is padding
    offsets = torch.tensor([0, 150, 151, wl.T], dtype=torch.int32, device=device)
    mask = torch.arange(wl.T, device=device) < wl.T - 20
    weight = mask.float() / mask.sum()

    history = {"distill": [], "reward": [], "balance": []}
    teacher_head = model.head.clone()
    model.head += 0.5 * wl.H ** -0.5 * torch.randn(model.head.shape, generator=g, device=device)
    top = model.teacher_top(x, teacher_head)
    for _ in range(distill_steps):
        z, saved = model.forward(x)
        loss, dz = M.distill_loss_grad(z, top[0], top[1], weight, teacher_lse=top[2], dlogits=z)
        losses, _ = model.step(saved, dz, offsets, mask, rate=1.0)
        history["distill"].append(float((loss * weight).sum()))
        history["balance"].append(float(losses[0]))

    # policy: tokens of the lower half of the vocabulary are rewarded
    for i in range(policy_steps):
        z, saved = model.forward(x)
        if i % 4 == 0:  # a new rollout every four updates
            actions = torch.multinomial(torch.softmax(z.float(), 1), 1, generator=g).squeeze(1)
            actions = torch.where(mask, actions, -1)  # padding has no token
            if i == 0:
                reference_z = z.clone()
            old, reference = M.token_logp(z, actions), M.token_logp(reference_z, actions)
            reward = (actions < VOCAB // 2).float()
            adv = reward - (reward * weight).sum()
        p_good = torch.softmax(z.float(), 1)[:, :VOCAB // 2].sum(1)
        history["reward"].append(float((p_good * weight).sum()))
        _, _, dz = M.policy_loss_grad(z, actions, old, adv, weight, ref_logp=reference,
                                      clip_high=0.28, kl_coef=0.01, dlogits=z)
        model.step(saved, dz, offsets, mask, rate=1.0)
    return history


if __name__ == "__main__":
    for name, values in run().items():
        print(name, " ".join(f"{v:.4f}" for v in values))
