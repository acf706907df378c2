"""Shared by the tests of the paged 8-bit cache: seeded batches on shuffled
pages, with NaN codes and NaN scales wherever a kernel must not look."""
import numpy as np

from diffusion_speculative_verification_gb300 import workloads as W
import oracle.paged as opaged


class PagedBatch:
    """Sequences (C, N, B), a shuffled page table with room for N + B more
    tokens each, K / V codes and scales, fresh rows; `pad` rows of NaN behind
    the last sequence, `idle` sequence indices with an idle record."""

    def __init__(self, C, N, B, Hq, Hkv, d, page, seed, dtype=W.BF16, pad=0, idle=(), spread=2, extra=3, qstd=1.0):
        r = np.random.default_rng(seed)
        C, N, B = (np.array(x, np.int64) for x in (C, N, B))
        self.Hq, self.Hkv, self.d, self.page, self.dtype = Hq, Hkv, d, page, dtype
        self.seqs = W.seq_table(C, N, B)
        need = -(-(C + N + B) // page)
        self.n_pages = int(need.sum()) + extra
        perm = r.permutation(self.n_pages).astype(np.int32)
        mp = max(1, int(need.max(initial=0)))
        self.table = np.full((len(C), mp), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.seqs[:, 4] = np.arange(len(C)) * mp
        self.tau = np.concatenate([W.random_tau(r, int(b)) for b in B]).astype(np.int32)
        self.n_acc = np.array([r.integers(0, b + 1) for b in B], np.int32)
        rows = int(np.sum(N + 2 * B))
        shape = (self.n_pages, Hkv, page, d)
        self.codes, self.scale = [], []
        for _ in range(2):
            codes = np.full(shape, 0x7F, np.uint8)
            scale = np.full((self.n_pages, Hkv), np.nan, np.float32)
            for b in range(len(C)):
                for j in range(-(-int(C[b]) // page)):
                    p, n = self.table[b, j], min(page, int(C[b]) - j * page)
                    x = r.standard_normal((Hkv, n, d)) * 2.0 ** r.integers(-spread, spread + 1)
                    for h in range(Hkv):
                        scale[p, h] = opaged.scale_for(float(np.abs(x[h]).max()))
                        codes[p, h, :n] = opaged.e4m3_codes(x[h] / scale[p, h])
            self.codes.append(codes)
            self.scale.append(scale)

        def fresh(h, std=1.0):
            x = W._store((r.standard_normal((rows + pad, h, d)) * std).astype(np.float32), dtype)
            x[rows:] = np.array(0x7FC0, np.uint16) if dtype == W.BF16 else np.nan
            return x

        self.q, self.k_new, self.v_new = fresh(Hq, qstd), fresh(Hkv), fresh(Hkv)
        for b in idle:
            self.seqs[b, :3] = 0
        self.rows, self.idle = rows, set(idle)

    def live(self):
        return [b for b in range(len(self.seqs)) if b not in self.idle]

    def values(self, x):
        return W.values_f64(x, self.dtype)

    def bounds(self):
        s = self.seqs
        return (len(self.tau), int(s[:, 0].max(initial=0)), int(s[:, 1].max(initial=0)),
                int(s[:, 2].max(initial=1)))

    def device(self, strided=False):
        """dict of device tensors; strided: fresh keys and values are parts of one buffer."""
        import torch
        from diffusion_speculative_verification_gb300 import ssv, io as sio
        t = dict(q=sio.tensor(self.q, self.dtype, "cuda"), tau=sio.int_tensor(self.tau, "cuda"),
                 pages=sio.int_tensor(self.table, "cuda"), n_acc=sio.int_tensor(self.n_acc, "cuda"))
        k, v = sio.tensor(self.k_new, self.dtype, "cuda"), sio.tensor(self.v_new, self.dtype, "cuda")
        if strided:
            buf = torch.full((k.shape[0], 2 * self.Hkv + 1, self.d), float("nan"), dtype=k.dtype, device="cuda")
            buf[:, :self.Hkv], buf[:, self.Hkv + 1:] = k, v
            k, v = buf[:, :self.Hkv], buf[:, self.Hkv + 1:]
        t["k_new"], t["v_new"] = k, v
        for i, x in enumerate("kv"):
            t[x + "_cache"] = torch.from_numpy(self.codes[i].copy()).cuda()
            t[x + "_scale"] = torch.from_numpy(self.scale[i].copy()).cuda()
        slots, mc, mn, mb = self.bounds()
        t["batch"] = ssv.Batch.from_device(sio.int_tensor(self.seqs, "cuda"), self.q.shape[0], slots, mc, mn, max(mb, 1))
        return t

    def caches(self):
        """Float64 caches laid out as oracle.attention wants them: (k, v, seqs with its kv_off)."""
        seqs = self.seqs.copy()
        parts = [[], []]
        at = 0
        for b in range(len(seqs)):
            seqs[b, 4] = at
            at += int(seqs[b, 0])
            for i in range(2):
                parts[i].append(opaged.gather_cache(self.seqs[b], self.table.reshape(-1), self.codes[i], self.scale[i]))
        return np.concatenate(parts[0]), np.concatenate(parts[1]), seqs
