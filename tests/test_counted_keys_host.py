"""The counting inputs of the fp8 attention's tests show every mistake they are meant to show: planted
here in the expected rows, on the host."""
import numpy as np
import pytest

from counted_keys import Counted


def as_bf16(x):
    """float64 -> nearest bf16 (ties to even), as float64."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("q_len,lengths,mask", [(1, [1, 2, 47, 48, 49, 97, 577], None), (9, [9, 48, 97, 385], True),
                                                (3, [20003, 6], True), (3, [29009], True), (1, [3000, 700, 1], None)])
def test_mistakes_show(q_len, lengths, mask):
    rng = np.random.default_rng(0)
    c = Counted(q_len, 8, lengths, seed=1, mask=mask)
    pool = c.table[c.table >= 0]
    for b in range(c.B):
        for t in range(q_len):
            s = c.keys(b, t)
            if not len(s):
                continue
            right = c.expected(s)
            assert c.agree(as_bf16(right[0]), np.float32(right[1]), *right)
            for _ in range(20):
                i = int(rng.integers(len(s)))
                wrong = [np.append(s, s[i])]                                        # taken twice
                if len(s) > 1:
                    wrong.append(np.delete(s, i))                                   # left out
                other = s.copy()
                other[i] = rng.choice(pool)                                         # from another slot
                if c.dim[other[i]] != c.dim[s[i]] or c.scale[other[i]] != c.scale[s[i]]:
                    wrong.append(other)
                for keys in wrong:
                    got = c.expected(keys)
                    assert not c.agree(as_bf16(got[0]), np.float32(got[1]), *right), (b, t, len(s), len(keys))
