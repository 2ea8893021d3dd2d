"""tokens_per_seq at the C boundary (no GPU: refused, or nothing to do)."""
from test_abi_paged import OK, SHAPE, attend, cache, gather, lib  # noqa: F401


def test_tokens_per_seq(lib):  # noqa: F811
    for tokens, want in ((0, OK), (1, OK), (4, OK), (2 ** 31 - 1, OK), (-1, SHAPE)):
        kv = cache()
        kv.tokens_per_seq = tokens
        assert attend(lib, kv=kv) == want
        assert gather(lib, kv=kv) == OK                 # of the attention alone
