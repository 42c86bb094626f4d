"""CPU: numbers of users at which the paged calls' 32-bit counters would wrap are refused before anything is
read or launched."""
from test_paged_abi import UNSUPPORTED, _append, _attn, lib  # noqa: F401  (lib: fixture)


def test_more_users_than_can_be_numbered(lib):
    """Items are numbered by H * (total_new / 128 + B); the scans step past B by a block's threads."""
    for users in ((1 << 30) + 1, 2 ** 31 - 100, 2 ** 31 - 1):
        assert _append(lib, B=users) == UNSUPPORTED, users
        for rows in (16, 2 ** 31 - 1):
            assert _attn(lib, B=users, total=rows, max_new=8) == UNSUPPORTED, (users, rows)
            assert _attn(lib, B=users, total=rows, max_new=rows, max_kv=2 ** 31 - 4097) == UNSUPPORTED, (users, rows)
