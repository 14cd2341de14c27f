"""What the attention's backward pass asks for in workspace, where first tokens
stay visible behind a window."""
import numpy as np
import pytest

from test_attention_host import Z  # noqa: F401  (fixture)


def test_first_tokens_cost_what_long_sequences_need(Z):  # noqa: F811
    """64 heads of 128 on 8, window 1024, 65536 tokens: at most one part of dk and dv (128 keys x 128 columns x 2 binary32, 128 KB
    a key head) for each 1152 tokens, and one for each 1024 queries and for what each such sequence has beyond."""
    plain = Z.attention_params(64, 8, 128, window=1024)
    sinks = Z.attention_params(64, 8, 128, window=1024, sinks=4)
    part = 2 * 128 * 128 * 4 * 8
    for n in (1, 16, 64, 1024, 20000):
        without, need = (Z.zero_attention_workspace_bytes(p, 65536, n) for p in (plain, sinks))
        long = 65536 // 1152
        assert without <= need <= without + part * (long + 64 + long) + 1024, n
    # no sequence can reach behind the window
    for tokens in (1, 500, 1151):
        assert Z.zero_attention_workspace_bytes(sinks, tokens, 3) == Z.zero_attention_workspace_bytes(plain, tokens, 3)


@pytest.mark.parametrize("window,sinks", [(1, 1), (70, 3), (128, 128), (1024, 16), (1 << 30, 4), ((1 << 32) - 2, 4), (70, 129)])
def test_holds_smaller_batches(Z, window, sinks):  # noqa: F811
    rng = np.random.default_rng(window % 1000 + sinks)
    for heads, kv, dim in ((2, 1, 64), (25, 25, 64), (64, 8, 128), (600, 600, 8)):
        p = Z.attention_params(heads, kv, dim, window=window, sinks=sinks)
        for most_tokens, most_n in ((9000, 1), (9000, 7), (3000, 300), (200, 2)):
            whole = Z.zero_attention_workspace_bytes(p, most_tokens, most_n)
            for tokens in {int(t) for t in rng.integers(1, most_tokens + 1, 60)} | {most_tokens}:
                for n in {1, 2, most_n, int(rng.integers(1, most_n + 1))}:
                    if n <= most_n:
                        assert Z.zero_attention_workspace_bytes(p, tokens, n) <= whole, (heads, tokens, n)
