"""A small hybrid decoder's layers over a prompt, single tokens and a speculative round.

Two layers of each kind, random weights, two requests:

  recurrent layer   conv + gated delta rule: gdn.conv_step and gdn.chunk_prefill over the prompt,
                    gdn.conv_decode_step for a token, gdn.conv_tree_verify and
                    gdn.conv_commit_path for a draft tree
  attention layer   gdn.kv_plan once a step, then gdn.kv_append and gdn.kv_attention over the
                    paged 8-bit cache, for all three

After a round the accepted path is committed: the recurrent layers replay it, and the cache's
lengths go back to the context and take the path's rows again (kv_append with ``rows``).

    python examples/hybrid_step.py        # needs a GB300 and the built library
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from hybrid_linear_attention_conv_gb300 import gdn  # noqa: E402

DEV = "cuda"
HK, HV, DK = 2, 6, 128          # recurrent layers: key heads, value heads, head size
HQ, HKV, D, PAGE = 12, 2, 256, 64  # attention layers
HIDDEN, LAYERS, REQUESTS, MAX_PAGES = 512, 2, 2, 16
C = gdn.packed_channels(HK, HV, DK, DK)


def _weight(g, n, m):
    return (torch.randn((n, m), generator=g, device=DEV) * n ** -0.5).to(torch.bfloat16)


class Hybrid:
    """The layers' weights and the requests' states: fixed-size ones, and the cache."""

    def __init__(self, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.w_in = [_weight(g, HIDDEN, C + 2 * HV) for _ in range(LAYERS)]
        self.w_conv = [(torch.randn((C, 4), generator=g, device=DEV) * 0.5).to(torch.bfloat16) for _ in range(LAYERS)]
        self.w_out = [_weight(g, HV * DK, HIDDEN) for _ in range(LAYERS)]
        self.w_qkv = [_weight(g, HIDDEN, (HQ + 2 * HKV) * D) for _ in range(LAYERS)]
        self.w_o = [_weight(g, HQ * D, HIDDEN) for _ in range(LAYERS)]
        # recurrent layers: state and conv tail (two buffers in turn) of each request
        self.state = torch.zeros((LAYERS, REQUESTS, HV, DK, DK), device=DEV)
        self.tail = torch.zeros((2, LAYERS, REQUESTS, 4, C), dtype=torch.bfloat16, device=DEV)
        self.turn = 0
        # attention layers: a cache each, pages and lengths in common
        pages = REQUESTS * MAX_PAGES
        f8 = torch.float8_e4m3fn
        self.cache = [(torch.empty((pages, HKV, PAGE, D), dtype=f8, device=DEV), torch.empty((pages, HKV, PAGE, D), dtype=f8, device=DEV),
                       torch.ones((pages, HKV), device=DEV), torch.ones((pages, HKV), device=DEV)) for _ in range(LAYERS)]
        i32 = dict(dtype=torch.int32, device=DEV)
        self.lens, self.held = torch.zeros(REQUESTS, **i32), torch.zeros(REQUESTS, **i32)
        self.free_pages = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        self.free_count = torch.tensor([pages], **i32)
        self.table = torch.full((REQUESTS, MAX_PAGES), -1, **i32)
        self.workspace = torch.zeros(gdn.kv_attention_workspace_bytes(HQ, HKV, D), dtype=torch.uint8, device=DEV)

    # ------------------------------------------------------------------ the two kinds of layer
    def project(self, i, x):
        """A recurrent layer's inputs: pre-conv rows, decay and write strength."""
        y = x @ self.w_in[i]
        alpha = torch.exp(-0.1 * torch.nn.functional.softplus(y[:, C:C + HV].float()))
        return y[:, :C].contiguous(), alpha, torch.sigmoid(y[:, C + HV:].float())

    def attention(self, i, x, plan, tree=None, keep=None):
        """An attention layer over the step's rows; `keep` collects its k and v rows."""
        lens, _, _, start, slots, _ = plan
        row = x @ self.w_qkv[i]
        q, k, v = (t.unflatten(1, (-1, D)) for t in row.split([HQ * D, HKV * D, HKV * D], dim=1))  # slices of the rows
        gdn.kv_append(k, v, slots, *self.cache[i])
        out = gdn.kv_attention(q, *self.cache[i], self.table, start, lens, tree=tree, workspace=self.workspace)
        if keep is not None:
            keep.append((q, k, v, out))
        return x + out.flatten(1) @ self.w_o[i]

    def plan(self, new, rows, keep=True):
        """Pages and slots for `new` tokens of each request; `keep`: the lengths move on."""
        new = torch.tensor(new, dtype=torch.int32, device=DEV)
        plan = gdn.kv_plan(self.lens, new, self.held, self.free_pages, self.free_count, self.table, PAGE, rows)
        gdn.kv_plan_check(plan[5])
        self.held, self.free_count = plan[1], plan[2]  # pages handed out stay with their request
        if keep:
            self.lens = plan[0]
        return plan

    # ------------------------------------------------------------------ the three kinds of step
    def prompt(self, xs, keep=None):
        """One prompt a request (rows of different lengths), into empty states."""
        n = [len(x) for x in xs]
        plan = self.plan(n, sum(n))
        x = torch.cat(xs)
        for i in range(LAYERS):
            u, alpha, beta = self.project(i, x)
            outs, at = [], 0
            for b in range(REQUESTS):
                part = slice(at, at + n[b])
                at += n[b]
                y = gdn.conv_step(u[None, part], self.w_conv[i], self.tail[self.turn, i, b:b + 1])
                outs.append(gdn.chunk_prefill(y[0], alpha[part].clone(), beta[part].clone(), self.state[i, b], HK, HV, DK, DK,
                                              out_bf16=True))
            x = x + torch.cat(outs).flatten(1) @ self.w_out[i]
            x = self.attention(i, x, plan, keep=keep)
        return x

    def token(self, x, keep=None):
        """One token of every request."""
        plan = self.plan([1] * REQUESTS, REQUESTS)
        for i in range(LAYERS):
            u, alpha, beta = self.project(i, x)
            o = gdn.conv_decode_step(u[:, None], self.w_conv[i], self.tail[self.turn, i], alpha[:, None], beta[:, None], self.state[i], HK,
                                     HV, DK, DK, tail_out=self.tail[1 - self.turn, i], out_bf16=True)
            x = x + o.flatten(1) @ self.w_out[i]
            x = self.attention(i, x, plan, keep=keep)
        self.turn = 1 - self.turn
        return x

    def verify(self, x, parents, keep=None):
        """A draft tree (parents [n]) of every request: rows [REQUESTS * n]; nothing is committed."""
        n = len(parents)
        masks = []
        for i, p in enumerate(parents):
            masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        tree = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks] * REQUESTS, dtype=torch.int64, device=DEV)
        plan = self.plan([n] * REQUESTS, REQUESTS * n, keep=False)
        drafts = []  # what a commit replays
        for i in range(LAYERS):
            u, alpha, beta = self.project(i, x)
            outs = []
            for b in range(REQUESTS):
                part = slice(b * n, (b + 1) * n)
                outs.append(gdn.conv_tree_verify(parents, u[part], self.w_conv[i], self.tail[self.turn, i, b], alpha[part].clone(),
                                                 beta[part].clone(), self.state[i, b], HK, HV, DK, DK, out_bf16=True))
            x = x + torch.cat(outs).flatten(1) @ self.w_out[i]
            kept = []
            x = self.attention(i, x, plan, tree=tree, keep=kept)
            drafts.append((u, alpha, beta, kept[0][1], kept[0][2]))
            if keep is not None:
                keep += kept
        return x, drafts

    def commit(self, parents, path, drafts):
        """The accepted root path (the same nodes of every request's tree)."""
        n = len(parents)
        plan = self.plan([len(path)] * REQUESTS, REQUESTS * len(path))  # from the context's length again
        rows = torch.tensor([b * n + node for b in range(REQUESTS) for node in path], dtype=torch.int32, device=DEV)
        for i, (u, alpha, beta, k, v) in enumerate(drafts):
            for b in range(REQUESTS):
                part = slice(b * n, (b + 1) * n)
                gdn.conv_commit_path(parents, path, u[part], self.w_conv[i], self.tail[self.turn, i, b], self.tail[1 - self.turn, i, b],
                                     alpha[part].clone(), beta[part].clone(), self.state[i, b], HK, HV, DK, DK)
            gdn.kv_append(k, v, plan[4], *self.cache[i], rows=rows)
        self.turn = 1 - self.turn


def run(seed=0):
    """A prompt, three tokens, a speculative round and a token after it.  The attention layers are
    compared with attention over unquantised keys and values on the same rows; returns the largest
    relative error of a step and layer (the cache's 8 bits), and the round's states against those of
    single tokens."""
    g = torch.Generator(device=DEV).manual_seed(100 + seed)
    new = lambda n: torch.randn((n, HIDDEN), generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    model = Hybrid(seed)
    history = [[[[], []] for _ in range(REQUESTS)] for _ in range(LAYERS)]
    errors = []

    def check(kept, counts, masks=None):
        """masks [n, n]: which of its own request's new rows a row sees (causal without)."""
        for i, (q, k, v, out) in enumerate(kept):
            at = 0
            for b, n in enumerate(counts):
                part = slice(at, at + n)
                at += n
                ks, vs = history[i][b]
                K, V = torch.cat(ks + [k[part].float()]), torch.cat(vs + [v[part].float()])
                seen = torch.ones((n, len(K)), dtype=torch.bool, device=DEV)
                seen[:, -n:] = torch.tril(seen[:, -n:]) if masks is None else masks
                a = torch.einsum("nhgd,lhd->hgnl", q[part].float().unflatten(1, (HKV, -1)), K) * D ** -0.5
                a = a.masked_fill(~seen, -torch.inf).softmax(-1)
                want = torch.einsum("hgnl,lhd->nhgd", a, V).flatten(1, 2)
                errors.append(float((out[part].float() - want).norm() / want.norm()))
                if masks is None:
                    ks.append(k[part].float())
                    vs.append(v[part].float())

    lengths = [150, 70]
    kept = []
    model.prompt([new(n) for n in lengths], keep=kept)
    check(kept, lengths)
    for _ in range(3):
        kept = []
        model.token(new(REQUESTS), keep=kept)
        check(kept, [1] * REQUESTS)

    parents, path = [-1, 0, 0, 1, 1, 2, 3, 5, 6], [0, 1, 3, 6]
    before = model.state.clone(), model.tail[model.turn].clone()
    seen = np.zeros((len(parents), len(parents)), bool)
    for i in range(len(parents)):
        m = i
        while m >= 0:
            seen[i, m] = True
            m = parents[m]
    kept = []
    x = new(REQUESTS * len(parents))
    _, drafts = model.verify(x, parents, keep=kept)
    check(kept, [len(parents)] * REQUESTS, torch.from_numpy(seen).to(DEV))
    model.commit(parents, path, drafts)
    for i, (_, k, v, _) in enumerate(kept):
        for b in range(REQUESTS):
            for node in path:
                history[i][b][0].append(k[b * len(parents) + node][None].float())
                history[i][b][1].append(v[b * len(parents) + node][None].float())

    # the committed recurrent states are those of the path's rows decoded one by one
    same = True
    for i, (u, alpha, beta, _, _) in enumerate(drafts):
        rows = [[b * len(parents) + node for b in range(REQUESTS)] for node in path]
        state, tail = before[0][i].clone(), before[1][i].clone()
        for r in rows:
            gdn.conv_decode_step(u[r][:, None].contiguous(), model.w_conv[i], tail, alpha[r][:, None].contiguous(),
                                 beta[r][:, None].contiguous(), state, HK, HV, DK, DK)
        same = same and torch.equal(state, model.state[i]) and torch.equal(tail, model.tail[model.turn, i])

    kept = []
    model.token(new(REQUESTS), keep=kept)
    check(kept, [1] * REQUESTS)
    lens = model.lens.tolist()
    assert lens == [n + 3 + len(path) + 1 for n in lengths], lens
    assert gdn.kv_attention_status(model.workspace) == 0
    return max(errors), same


if __name__ == "__main__":
    error, same = run()
    print(f"attention over the 8-bit cache: largest relative error of a layer's output {error:.3f}; "
          f"committed states equal single tokens': {same}")
