"""Inputs of mla_verify_attn_fp8 that count its keys: queries of zero, so that all scores are equal, and
keys with a single non-zero code at one dim, so that each output dim is the sum of its keys' scales over
the number of keys and the log-sum-exp that number's logarithm."""
import numpy as np

import step_ref as ref

ONE = 0x38                         # the e4m3 code of 1.0


class Counted:
    def __init__(self, q_len, H, lengths, *, seed, mask=None, extra_stride=0):
        rng = np.random.default_rng(seed)
        self.B, self.q_len, self.H, self.seq = len(lengths), q_len, H, np.array(lengths, np.int32)
        total = int(self.seq.sum())
        n_pool = total + 5
        perm = rng.permutation(n_pool).astype(np.int32)
        self.table = np.full((self.B, int(self.seq.max()) + extra_stride), -1, np.int32)
        first = np.cumsum(self.seq) - self.seq
        for b in range(self.B):
            self.table[b, :self.seq[b]] = perm[first[b]:first[b] + self.seq[b]]
        self.dim = rng.integers(0, 512, n_pool)
        self.scale = (2.0 ** rng.integers(0, 3, n_pool)).astype(np.float32)
        self.lat = np.zeros((n_pool, 512), np.uint8)
        self.lat[np.arange(n_pool), self.dim] = ONE
        unused = perm[total:]
        self.lat[unused], self.scale[unused] = 0x7F, np.nan
        self.rope = rng.normal(size=(n_pool, 64)).astype(np.float32)
        self.rope[unused] = np.nan
        self.mask = (rng.random((self.B, q_len, q_len)) < 0.5).astype(np.uint8) if mask else None

    def keys(self, b, t):
        """The slots that draft t of stream b sees."""
        n = int(self.seq[b])
        return self.table[b, :n][ref.visible(self.mask, b, t, n, self.q_len)]

    def expected(self, slots):
        """(out [512], lse) of a row that sees these slots."""
        return (np.bincount(self.dim[slots], weights=self.scale[slots].astype(np.float64), minlength=512) / len(slots),
                np.log(len(slots)))

    @staticmethod
    def agree(out, lse, want_out, want_lse):
        """The weights are exact powers of two and their sums whole numbers below 2^24; what rounds are two
        logarithms, 1 / l, the merge's weights (fp32, a few steps of 2^-24 of numbers up to 32) and the
        output in bf16."""
        return bool(np.all(np.abs(out - want_out) <= want_out * (ref.BF16_HALF + 2.0 ** -17)) and
                    np.all(np.abs(lse - want_lse) <= 2.0 ** -17))
