"""How kv4_attention cuts sessions into shares, restated on the CPU in the kernel's own integer steps: every chunk of
every session is taken once, and the records that the join goes by name the blocks whose partial results make up a unit."""
import random

import pytest

START = 20                  # places that a session's start counts as
U32, SMALL = (1 << 32) - 1, 1 << 31


def pieces(chunks, shares, share, least, wrap=False):
    """The pieces of one share: (session, chunk0, chunk1, share0, sharers, late).  wrap: the share's length is cut to 32
    bits as it stands, not limited to them."""
    total = sum(START + c for c in chunks) - START
    q = max((total + shares - 1) // shares, least)
    pos, end = share * q, min(share * q + q, total)
    session, before, run = None, None, -START
    for s, c in enumerate(chunks):
        if run <= pos < run + START + c:
            session, before = s, run
        run += START + c
    out = []
    while pos < end:
        first, n = before + START, chunks[session]
        if end <= first:
            break
        if first + n < SMALL:
            q32 = q & U32 if wrap else min(q, U32)
            share0, share1 = first // q32, (first + n - 1) // q32
        else:
            share0, share1 = first // q, (first + n - 1) // q
        chunk0, chunk1 = max(pos - first, 0), min(n, end - first)
        out.append((session, chunk0, chunk1, share0, share1 - share0 + 1, before > share0 * q))
        pos = first + chunk1
        if chunk1 == n:
            before, session = pos, session + 1
    return out


def check(chunks, shares, least, wrap=False):
    cut = [pieces(chunks, shares, k, least, wrap) for k in range(shares)]
    upto = [0] * len(chunks)
    joined = {}                                  # session: (share0, sharers, late) of its record
    for k, share in enumerate(cut):
        for i, (s, a, b, share0, sharers, late) in enumerate(share):
            assert a == upto[s] and a < b <= chunks[s]
            upto[s] = b
            assert share0 <= k < share0 + sharers
            assert (sharers == 1) == (a == 0 and b == chunks[s])
            if sharers > 1 and share0 == k:
                assert s not in joined and i == len(share) - 1      # a share's last piece, one record a share
                joined[s] = share0, sharers, late
    assert upto == chunks
    for s, (share0, sharers, late) in joined.items():
        for k in range(share0, share0 + sharers):                   # each of them has a piece of it
            at = [i for i, p in enumerate(cut[k]) if p[0] == s]
            assert len(at) == 1
            # the join reads the partial of the share's first piece, or of its last if that starts late in share0
            assert (k == share0 and late) or at[0] == 0 or not any(p[4] > 1 for p in cut[k][:at[0]])
            if k > share0:
                assert at[0] == 0
    for k, share in enumerate(cut):                                 # two partials of a share do not share a place
        slots = [p[3] == k and p[5] for p in share if p[4] > 1]
        assert len(slots) == len(set(slots))


@pytest.mark.parametrize("seed", range(6))
def test_every_chunk_is_taken_once(seed):
    rnd = random.Random(seed)
    for _ in range(150):
        top = rnd.choice((1, 3, 40, 300, 3000))
        chunks = [rnd.randrange(1, top + 1) for _ in range(rnd.choice((1, 2, 7, 40, 300)))]
        check(chunks, rnd.choice((1, 2, 19, 38, 152, 304)), rnd.choice((6, 8)))


def test_more_places_than_32_bits_hold():
    chunks = [1 << 26] * 64 + [5, 1 << 26, 1]
    for shares in (1, 2, 304):
        check(chunks, shares, 8)
    with pytest.raises(AssertionError):
        check(chunks, 1, 8, wrap=True)
