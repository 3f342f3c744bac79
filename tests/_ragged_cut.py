"""How decode_tree cuts its work, restated from the sizes, so that tests can say which way they take.

CTAs work in teams of one per block of 2 * floor(128 / G) drafted tokens of the longest row. A unit is
one (row, KV head), or several KV heads of a row with fewer blocks; it has a tile per 128 context slots
and one for the drafted tokens. Units are not cut when the cache has at most 4 tiles ("whole"). Else the
teams take one part each when equal parts of at most ceil(all tiles / teams) tiles are not more than
there are teams ("even"), and otherwise equal shares of all units in one line ("line").
"""


def _cdiv(a, b):
    return -(-a // b)


def cut(contexts, drafts, S_max, H_q, H_kv, max_tokens, sms):
    """Returns (way, teams, parts of the longest row's units when cut evenly)."""
    G = H_q // H_kv
    tok = 128 // G
    team = 1 if max_tokens <= tok else _cdiv(max_tokens, 2 * tok)
    row_tiles = _cdiv(S_max, 128) + 1
    most = max(1, min(sms, 152) // team)
    if row_tiles <= 5:
        return "whole", min(len(drafts) * H_kv, most), 1
    teams = min(len(drafts) * H_kv * row_tiles, most)
    units = []
    for c, t in zip(contexts, drafts):
        if t:
            blocks = 1 if team == 1 else _cdiv(t, 2 * tok)
            units += [_cdiv(c, 128) + 1] * _cdiv(H_kv, team // blocks)
    longest = max(1, _cdiv(sum(units), teams))
    parts = [_cdiv(u, longest) for u in units]
    return ("even" if sum(parts) <= teams else "line"), teams, max(parts, default=1)
