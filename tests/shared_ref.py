"""Batches of sequences with common prefixes, over caches of every kind, and
attention over them in float64 with what a correct kernel may be off by."""
import numpy as np
import torch

import paged_attention_decode_split_gb300 as pa
from tests import fp4_ref

KINDS = ["bf16", "fp8", "fp4"]


def e4m3(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).float().numpy()


class Batch:
    """groups: per group (prefix tokens, [tokens of each sequence beyond it; None = idle])."""

    def __init__(self, seed, groups, hq, hkv, d, bs, kind="bf16", out="f32"):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.bs, self.kind, self.out = hq, hkv, d, bs, kind, out
        lens, prefix, starts = [], [], [0]
        for pre, own in groups:
            for n in own:
                lens.append(0 if n is None else pre + n)
                prefix.append(pre)
            starts.append(len(lens))
        self.lens, self.prefix, self.starts = (np.array(x, np.int32) for x in (lens, prefix, starts))
        self.n = len(lens)
        self.width = max(1, -(-int(self.lens.max(initial=1)) // bs))
        self.pages = int(sum(-(-n // bs) for n in lens)) + 3
        order, at = rng.permutation(self.pages), 0
        self.table = np.full((self.n, self.width), -7, np.int32)
        copies = []  # (sequence, leader, page): a prefix that ends inside a page has its part of it copied
        for g, (pre, own) in enumerate(groups):
            leader = None
            for b in range(starts[g], starts[g + 1]):
                used = -(-lens[b] // bs)
                first = pre // bs if leader is not None and used else 0
                if lens[b] == 0:
                    continue
                self.table[b, first:used] = order[at:at + used - first]
                at += used - first
                if leader is None:
                    leader = b
                    continue
                self.table[b, :first] = self.table[leader, :first]
                if pre % bs >= 16 and first < used:
                    copies.append((self.table[b, first], self.table[leader, first], pre % bs // 16 * 16))
        self.k, self.v, self.g = self._caches(rng)
        for to, at, tokens in copies:
            for c in (self.k, self.v):
                if kind == "fp4":
                    c[to, :, :tokens // 16] = c[at, :, :tokens // 16]
                else:
                    c[to, :tokens] = c[at, :tokens]
        self.scale = 1 / np.sqrt(d)
        self.q = torch.from_numpy(rng.standard_normal((self.n, hq, d)).astype(np.float32)).to(torch.bfloat16)

    def _caches(self, rng):
        p, bs, hkv, d = self.pages, self.bs, self.hkv, self.d
        if self.kind == "fp4":
            g = fp4_ref.head_scales(hkv)
            return *fp4_ref.random_cache(rng, p, bs, hkv, d, g), g
        x = [torch.from_numpy(rng.standard_normal((p, bs, hkv, d)).astype(np.float32)) for _ in range(2)]
        if self.kind == "bf16":
            return x[0].to(torch.bfloat16), x[1].to(torch.bfloat16), None
        h = np.arange(hkv, dtype=np.float32)
        g = ((1 + h / 4) / 64).astype(np.float32), ((1 + h / 8) / 48).astype(np.float32)
        codes = [(t.clamp(-6, 6) / torch.from_numpy(s)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                 for t, s in zip(x, g)]
        return *codes, g

    def slots(self, b):
        """Where the tokens of sequence b stand."""
        t = np.arange(self.lens[b])
        return self.table[b].astype(np.int64)[t // self.bs] * self.bs + t % self.bs

    def rows(self, which, slots):
        c = (self.k, self.v)[which]
        if self.kind == "fp4":
            return fp4_ref.read_rows("kv"[which], c, slots, self.g[which])
        if self.kind == "bf16":
            return c.flatten(0, 1)[torch.from_numpy(slots)].double().numpy()
        return e4m3(c.reshape(-1, self.hkv, self.d)[slots]).astype(np.float64) * self.g[which].astype(np.float64)[:, None]

    def reference(self, f16_end=2.0 ** -24):
        """(outputs, tolerance): float64 [n, hq, d]; f16_end: of the largest weight, what f16 may lose of any."""
        ref, tol = np.zeros((self.n, self.hq, self.d)), np.zeros((self.n, self.hq, self.d))
        grp, q = self.hq // self.hkv, self.q.double().numpy()
        for b in range(self.n):
            if self.lens[b] == 0:
                continue
            s = self.slots(b)
            k, v = self.rows(0, s), self.rows(1, s)
            for h in range(self.hkv):
                hs = slice(h * grp, (h + 1) * grp)
                x = q[b, hs] @ k[:, h].T * self.scale
                reach = (np.abs(q[b, hs]) @ np.abs(k[:, h]).T).max(-1) * self.scale
                w = np.exp(x - x.max(-1, keepdims=True))
                total = w.sum(-1, keepdims=True)
                o, mag = w / total @ v[:, h], w / total @ np.abs(v[:, h])
                # A score is d products summed in binary32 (one step each, the tensor core may cut off): off by e; a
                # weight by a factor of 1 +- 1.01 e, by exp2 (2^-22) and by the two numbers it enters the product as
                # (bf16 head and residual: 2^-18; f16: 2^-22, or one f16 for bf16 outputs over fp4: 2^-11), and so is
                # their sum; the sums over keys lose a step (2^-23) per 16-key product and per merge.
                e = (self.d + 4) * 2.0 ** -23 * reach
                weight = 2.0 ** -17 if self.kind == "bf16" else 2.0 ** -11 if self.kind == "fp4" and self.out == "bf16" else 2.0 ** -21
                rel = 2.02 * e + 2 * (weight + 2.0 ** -22) + (len(s) / 16 + 64) * 2.0 ** -23
                # f16 ends at 2^-25: weights relative to a reference that gives the largest 1 or more
                lost = np.minimum(w, f16_end) / total @ np.abs(v[:, h]) if self.kind != "bf16" else 0.0
                ref[b, hs], tol[b, hs] = o, rel[:, None] * mag + lost + 1e-30
        return ref, tol + (np.abs(ref) * 2.0 ** -8 if self.out == "bf16" else 0.0)

    # -- the call ------------------------------------------------------------------

    def tensors(self):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
        put = lambda c: c.cuda() if isinstance(c, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(c)).cuda()  # noqa: E731
        scales = () if self.g is None else (put(self.g[0]), put(self.g[1]))
        return dict(q=self.q.cuda(), caches=(put(self.k), put(self.v)), scales=scales, table=i32(self.table).reshape(self.table.shape),
                    lens=i32(self.lens), starts=i32(self.starts), prefix=i32(self.prefix))

    def desc(self, num_splits=0, **kw):
        return pa.make_desc(**(dict(
            num_seqs=self.n, num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d, block_size=self.bs,
            max_pages_per_seq=self.width, max_seq_len=int(self.width * self.bs), num_pages=self.pages, scale=self.scale,
            out_dtype=pa.PA_OUT_BF16 if self.out == "bf16" else pa.PA_OUT_F32, num_splits=num_splits) | kw))

    def shared(self, **kw):
        size = int(np.diff(self.starts).max())
        return pa.make_prefix(**(dict(num_groups=len(self.starts) - 1, max_group_seqs=max(1, size),
                                      max_prefix_len=int(self.prefix.max()),
                                      max_suffix_len=max(1, int((self.lens - self.prefix).max()))) | kw))

    def run(self, t=None, desc=None, shared=None, workspace=None, status=None, out=None, stream=None, **kw):
        t, desc, shared = t or self.tensors(), desc or self.desc(), shared or self.shared(**kw)
        if out is None:
            out = torch.full((self.n, self.hq, self.d), float("nan"), device="cuda",
                             dtype=torch.bfloat16 if self.out == "bf16" else torch.float32)
        if workspace is None:
            workspace = torch.full((pa.shared_workspace_bytes(desc, shared),), 0xFF, dtype=torch.uint8, device="cuda")
        call = getattr(pa, "paged_attention_decode_shared" + ("" if self.kind == "bf16" else "_" + self.kind))
        call(t["q"], *t["caches"], *t["scales"], t["table"], t["lens"], t["starts"], t["prefix"], desc, shared, out, workspace,
             status=status, stream=stream)
        return out


def check(got, ref, tol):
    g = got.detach().double().cpu().numpy()
    assert np.isfinite(g).all()
    worst = np.max(np.abs(g - ref) / np.maximum(tol, 1e-300), initial=0.0)
    assert (np.abs(g - ref) <= tol).all(), f"{worst:.3g} times the tolerance"
    assert (g[tol == 0] == 0).all()  # idle sequences
