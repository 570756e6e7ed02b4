"""What the size queries answer where the calls themselves refuse (no GPU needed)."""
from test_more_ops_host import NULL, S, T, U, gar, tables  # noqa: F401


def test_rows_of_what_the_sort_refuses(gar):  # noqa: F811
    lib, (c, p) = gar.load(), tables(1, 0x1000000, 0x2000000)

    def sort(tokens, k, experts, align, capacity):
        return lib.gar_expert_sort(c, 1, tokens, k, experts, align, capacity, p, S, (1 << 31) - 1, T, U, 1 << 20, NULL)

    for args in ((1 << 30, 2, 8, 1, 0), ((1 << 25) + 1, 32, 8, 1, 0), (10, 2, 8, 2, 4), (10, 2, 1024, 1 << 22, 0), (10, 2, 1024, 1, 1 << 22)):
        assert sort(*args) == gar.GAR_EINVAL and lib.gar_expert_rows(1, *args) == -1, args
    assert lib.gar_expert_rows(1, 1 << 25, 32, 8, 1, 0) == 1 << 30
    assert lib.gar_expert_rows(1, 10, 2, 1024, 1, (1 << 21) - 1) == 1024 * ((1 << 21) - 1)


def test_workspace_of_what_the_vocabulary_layer_refuses(gar):  # noqa: F811
    f = gar.load().gar_vocab_workspace_bytes
    for rows, vocab, hidden in ((1 << 31, 100, 64), (1 << 62, 100, 64), (5, 1 << 31, 64), (5, 100, (1 << 20) + 1)):
        assert f(rows, vocab, hidden, 0) == 0
    assert f(5, 100, 1 << 20, 0) > 0
