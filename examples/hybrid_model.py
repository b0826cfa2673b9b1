"""A small language model around the fast-weight layer, trained and served on the
framework's operators.

Each block is two residual branches in pre-norm form:
  h += W_out mix(W_mix norm(h))   the gated linear recurrence as token mixer, or causal
                                  attention in the blocks listed in `attend`
  h += mlp(norm(h))               the gated feed-forward block, or the fast-weight
                                  layer in the blocks listed in `fast`
The residual add of a branch runs inside the next norm. Projections and the
embedding are plain torch products. Everything is bf16 with fp32 states, updated
by SGD on fp32 copies.

  python examples/hybrid_model.py      trains a few steps on packed synthetic
                                       documents, then decodes from a prompt
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunked_weight_mlp_amd import Layer, attention, block  # noqa: E402

BF16 = torch.bfloat16


class HybridModel:
    def __init__(self, vocab=256, d=128, d_ff=256, blocks=2, fast=(1,), chunk=64, max_batch=2,
                 max_seq_len=512, eta=1e-3, device="cuda", seed=0, attend=(), heads=4, k_heads=2):
        g = torch.Generator().manual_seed(seed)
        self.d, self.chunk, self.fast, self.blocks, self.eta = d, chunk, set(fast), blocks, eta
        self.max_batch, self.max_seq_len, self.device = max_batch, max_seq_len, device
        self.attend, self.hq, self.hk, self.dh = set(attend), heads, k_heads, d // heads

        def draw(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device)

        # fp32 parameters by name; the operators read bf16 copies
        p = {"embed": draw(vocab, d, std=1.0), "final.gamma": torch.ones(d, device=device),
             "final.beta": torch.zeros(d, device=device)}
        for i in range(blocks):
            for n in ("mix", "mlp"):
                p[f"{i}.{n}.gamma"] = torch.ones(d, device=device)
                p[f"{i}.{n}.beta"] = torch.zeros(d, device=device)
            if i in self.attend:
                p[f"{i}.w_mix"] = draw((heads + 2 * k_heads) * self.dh, d, std=d ** -0.5)
                for n in ("q_gamma", "k_gamma"):
                    p[f"{i}.{n}"] = torch.ones(self.dh, device=device)
            else:
                p[f"{i}.w_mix"] = draw(2 * d, d, std=d ** -0.5)
            p[f"{i}.w_out"] = draw(d, d, std=0.5 * d ** -0.5)
            p[f"{i}.w_gate"], p[f"{i}.w_up"] = draw(d_ff, d, std=d ** -0.5), draw(d_ff, d, std=d ** -0.5)
            p[f"{i}.w_down"] = draw(d, d_ff, std=0.5 * d_ff ** -0.5)
            if i in self.fast:
                p[f"{i}.proj"], p[f"{i}.conv_w"] = draw(d, d, std=d ** -0.5), draw(d, 4, std=0.5)
        self.params = p
        self.refresh()

    def refresh(self):
        """The operators over the parameters' current values."""
        w = self.w = {k: v.to(BF16) for k, v in self.params.items()}
        self.norms = {k[: -len(".gamma")]: block.Norm(w[k], w[k[: -len("gamma")] + "beta"])
                      for k in w if k.endswith(".gamma")}
        inv_freq = 1e4 ** (-torch.arange(0, self.dh, 2, dtype=torch.float64, device=self.device) / self.dh)
        self.head_norms = {i: attention.HeadNorm(w[f"{i}.q_gamma"], w[f"{i}.k_gamma"], inv_freq)
                           for i in self.attend}
        self.mlps = {}
        for i in range(self.blocks):
            if i in self.fast:
                # the pretrained down projection is the state's starting point, fp32
                self.mlps[i] = Layer(w_gate=w[f"{i}.w_gate"], w_up=w[f"{i}.w_up"], proj=w[f"{i}.proj"],
                                     conv_w=w[f"{i}.conv_w"], w0=self.params[f"{i}.w_down"].contiguous(),
                                     chunk=self.chunk, eta=self.eta, max_batch=self.max_batch,
                                     max_seq_len=self.max_seq_len)
            else:
                self.mlps[i] = block.FeedForward(w[f"{i}.w_gate"], w[f"{i}.w_up"], w[f"{i}.w_down"])

    def _heads(self, qkv):
        """Queries, keys and values of a fused projection, [tokens, heads, dh] each."""
        n = qkv.shape[-1] // self.dh
        return qkv.view(-1, n, self.dh).split([self.hq, self.hk, self.hk], 1)

    # ---- training ----------------------------------------------------------------------

    def loss_and_grads(self, tokens, targets, starts=None):
        """tokens, targets: [batch, seq_len]; starts marks packed documents for the token
        mixer (the fast weight runs over the whole row). Returns the mean cross entropy
        and the gradient of every parameter."""
        d, w = self.d, self.w
        e = w["embed"][tokens].contiguous()
        h, res, saved = e, None, []
        if self.attend:
            # the rows one after another: a sequence at each row's and each document's beginning
            first = torch.zeros(tokens.shape, dtype=torch.bool, device=self.device)
            first[:, 0] = True
            first = (first if starts is None else first | (starts != 0)).flatten()
            begin = first.nonzero()[:, 0]
            offsets = torch.cat([begin, begin.new_tensor([first.numel()])]).to(torch.int32)
            pos = (torch.arange(first.numel(), device=self.device)
                   - begin[first.cumsum(0) - 1]).to(torch.int32)
        for i in range(self.blocks):
            y1, h1, m1, r1 = self.norms[f"{i}.mix"].forward(h, res)
            gv = y1 @ w[f"{i}.w_mix"].t()
            if i in self.attend:
                q, k, v = self._heads(gv)
                qr, kr = self.head_norms[i].forward(q, k, pos)
                o, lse = attention.attention_forward(qr, kr, v, offsets=offsets)
                s, seen = o.view(tokens.shape + (d,)), (q, k, v, qr, kr, o, lse)
            else:
                s, _ = block.recurrence_forward(gv[..., :d], gv[..., d:], starts=starts)
                seen = None
            y2, h2, m2, r2 = self.norms[f"{i}.mlp"].forward(h1, s @ w[f"{i}.w_out"].t())
            mlp, a, u = self.mlps[i], None, None
            if i in self.fast:
                mlp.reset()
                res = mlp.prefill(y2, e).to(BF16)
            else:
                res, a, u = mlp.forward(y2, save=True)
            saved.append((y1, h1, m1, r1, gv, s, y2, h2, m2, r2, a, u, seen))
            h = h2
        y, hf, mf, rf = self.norms["final"].forward(h, res)
        logits = (y.float() @ w["embed"].float().t())
        logp = torch.log_softmax(logits, -1)
        loss = -logp.gather(-1, targets[..., None]).mean()

        dlogits = logp.exp()
        dlogits.scatter_add_(-1, targets[..., None], torch.full_like(dlogits[..., :1], -1.0))
        dlogits /= targets.numel()
        grads = {"embed": dlogits.flatten(0, 1).t() @ y.float().flatten(0, 1)}
        dy = (dlogits @ w["embed"].float()).to(BF16)
        g = self.norms["final"].backward(hf, mf, rf, dy)
        grads["final.gamma"], grads["final.beta"] = g["dgamma"], g["dbeta"]
        dh = g["dx"]              # gradient of the residual stream and of the last branch
        de = torch.zeros_like(e, dtype=torch.float32)
        for i in reversed(range(self.blocks)):
            y1, h1, m1, r1, gv, s, y2, h2, m2, r2, a, u, seen = saved[i]
            mlp = self.mlps[i]
            if i in self.fast:
                g = mlp.backward(y2, e, dh.float())
                de += g["de"]
                for n, k in (("w_gate", "dw_gate"), ("w_up", "dw_up"), ("w_down", "dw0"),
                             ("proj", "dproj"), ("conv_w", "dconv_w")):
                    grads[f"{i}.{n}"] = g[k]
                dy2 = g["dx"].to(BF16)
            else:
                g = mlp.backward(y2, a, u, dh)
                for n in ("w_gate", "w_up", "w_down"):
                    grads[f"{i}.{n}"] = g["d" + n].float()
                dy2 = g["dx"]
            g = self.norms[f"{i}.mlp"].backward(h2, m2, r2, dy2, dh)
            grads[f"{i}.mlp.gamma"], grads[f"{i}.mlp.beta"] = g["dgamma"], g["dbeta"]
            dh = g["dx"]
            flat = dh.flatten(0, 1)
            grads[f"{i}.w_out"] = flat.float().t() @ s.float().flatten(0, 1)
            ds = dh @ w[f"{i}.w_out"]
            dgv = torch.empty_like(gv)
            if i in self.attend:
                q, k, v, qr, kr, o, lse = seen
                g = attention.attention_backward(qr, kr, v, o, lse, ds.view_as(o), offsets=offsets)
                n = self.head_norms[i].backward(q, k, pos, g["dq"], g["dk"])
                grads[f"{i}.q_gamma"], grads[f"{i}.k_gamma"] = n["dq_gamma"], n["dk_gamma"]
                for part, grad in zip(self._heads(dgv), (n["dq"], n["dk"], g["dv"])):
                    part.copy_(grad)
            else:
                block.recurrence_backward(gv[..., :d], gv[..., d:], s, ds, starts=starts, dg=dgv[..., :d],
                                          dv=dgv[..., d:])
            grads[f"{i}.w_mix"] = dgv.float().flatten(0, 1).t() @ y1.float().flatten(0, 1)
            g = self.norms[f"{i}.mix"].backward(h1, m1, r1, dgv @ w[f"{i}.w_mix"], dh)
            grads[f"{i}.mix.gamma"], grads[f"{i}.mix.beta"] = g["dgamma"], g["dbeta"]
            dh = g["dx"]
        de += dh.float()
        grads["embed"].index_add_(0, tokens.flatten(), de.flatten(0, 1))
        return loss, grads

    def step(self, tokens, targets, starts=None, lr=0.3):
        loss, grads = self.loss_and_grads(tokens, targets, starts)
        for k, g in grads.items():
            self.params[k] -= lr * g
        self.refresh()
        return float(loss)

    # ---- serving -----------------------------------------------------------------------

    def prefill(self, tokens):
        """Runs prompts [batch, seq_len] of whole chunks; returns the logits of every token
        and keeps the states for decode()."""
        if tokens.shape[1] % self.chunk:
            raise ValueError("prompts are whole chunks: the fast weight's next chunk starts after them")
        if self.attend and tokens.shape[1] > self.max_seq_len:
            raise ValueError(f"{tokens.shape[1]} tokens do not fit the caches' max_seq_len={self.max_seq_len}")
        d, w = self.d, self.w
        e = w["embed"][tokens].contiguous()
        self.states, h, res = {}, e, None
        batch, length = tokens.shape
        self.length = length
        if self.attend:
            # a page table for max_seq_len tokens a sequence, which every block's cache shares
            page = 16
            width = -(-self.max_seq_len // page)
            self.table = torch.arange(batch * width, dtype=torch.int32, device=self.device).view(batch, width)
            self.lens = torch.full((batch,), length, dtype=torch.int32, device=self.device)
            seqs = torch.arange(batch, dtype=torch.int32, device=self.device).repeat_interleave(length)
            pos = torch.arange(length, dtype=torch.int32, device=self.device).repeat(batch)
            offsets = torch.arange(batch + 1, dtype=torch.int32, device=self.device) * length
            self.caches = {i: attention.KVCache.empty(batch * width, self.hk, page, self.dh, BF16, self.device)
                           for i in self.attend}
        for i in range(self.blocks):
            y, h, _, _ = self.norms[f"{i}.mix"].forward(h, res)
            gv = y @ w[f"{i}.w_mix"].t()
            if i in self.attend:
                q, k, v = self._heads(gv)
                self.head_norms[i].append(q, k, v, pos, self.caches[i], self.table, seqs)
                qr, kr = self.head_norms[i].forward(q, k, pos)
                s = attention.attention_forward(qr, kr, v, offsets=offsets)[0].view(batch, length, d)
            else:
                s, self.states[i] = block.recurrence_forward(gv[..., :d], gv[..., d:])
            y, h, _, _ = self.norms[f"{i}.mlp"].forward(h, s @ w[f"{i}.w_out"].t())
            if i in self.fast:
                self.mlps[i].reset()
                res = self.mlps[i].prefill(y, e).to(BF16)
            else:
                res = self.mlps[i].forward(y)
        self.pos = 0
        # the fast-weight layers' chunk in progress
        self.chunk_x = {i: torch.zeros(batch, self.chunk, d, dtype=BF16, device=self.device)
                        for i in self.fast}
        self.chunk_e = torch.zeros(batch, self.chunk, d, dtype=BF16, device=self.device)
        return self.norms["final"].forward(h, res)[0] @ w["embed"].t()

    def decode(self, tokens):
        """One token [batch] after the prefill or the last decode; returns its logits."""
        # a token behind the table's last page would not be written, nor attended to
        if self.attend and self.length >= self.max_seq_len:
            raise ValueError(f"the caches hold max_seq_len={self.max_seq_len} tokens a sequence already")
        self.length += 1
        d, w = self.d, self.w
        e = w["embed"][tokens].contiguous()
        self.chunk_e[:, self.pos] = e
        h, res = e, None
        for i in range(self.blocks):
            y, h, _, _ = self.norms[f"{i}.mix"].forward(h, res)
            gv = y @ w[f"{i}.w_mix"].t()
            if i in self.attend:
                q, k, v = self._heads(gv)
                qr = self.head_norms[i].append(q, k, v, self.lens, self.caches[i], self.table)
                s = attention.attention_step(qr, self.caches[i], self.table, self.lens + 1).view(-1, d)
            else:
                s, _ = block.recurrence_step(gv[:, :d], gv[:, d:], self.states[i], out=self.states[i])
            y, h, _, _ = self.norms[f"{i}.mlp"].forward(h, s @ w[f"{i}.w_out"].t())
            if i in self.fast:
                self.chunk_x[i][:, self.pos] = y
                res = self.mlps[i].decode_step(self.chunk_x[i], self.chunk_e, self.pos).to(BF16)
            else:
                res = self.mlps[i].forward(y)
        self.pos = (self.pos + 1) % self.chunk
        if self.attend:
            self.lens += 1
        return self.norms["final"].forward(h, res)[0] @ w["embed"].t()


def documents(batch, seq_len, vocab, seed, device="cuda"):
    """Packed synthetic documents: arithmetic progressions modulo the vocabulary, a new
    start and step per document. Returns tokens, targets and the document starts."""
    g = torch.Generator().manual_seed(seed)
    t = torch.zeros(batch, seq_len + 1, dtype=torch.long)
    starts = torch.zeros(batch, seq_len + 1, dtype=torch.uint8)
    for b in range(batch):
        at = 0
        while at <= seq_len:
            n = int(torch.randint(24, 96, (1,), generator=g))
            first, inc = (int(torch.randint(0, vocab, (1,), generator=g)),
                          int(torch.randint(1, 4, (1,), generator=g)))
            m = min(n, seq_len + 1 - at)
            t[b, at:at + m] = (first + inc * torch.arange(m)) % vocab
            starts[b, at] = 1
            at += n
    t, starts = t.to(device), starts.to(device)
    return t[:, :-1].contiguous(), t[:, 1:].contiguous(), starts[:, :-1].contiguous()


def main():
    model = HybridModel()
    for k in range(30):
        tokens, targets, starts = documents(2, 512, 256, seed=k)
        loss = model.step(tokens, targets, starts)
        if k % 5 == 0 or k == 29:
            print(f"step {k}: loss {loss:.3f}", flush=True)
    tokens, _, _ = documents(2, 128, 256, seed=1000)
    logits = model.prefill(tokens)
    nxt = logits[:, -1].argmax(-1)
    out = [nxt]
    for _ in range(15):
        nxt = model.decode(nxt).argmax(-1)
        out.append(nxt)
    print("prompt ends", tokens[:, -4:].tolist(), "decoded", torch.stack(out, 1).tolist(), flush=True)


if __name__ == "__main__":
    main()
