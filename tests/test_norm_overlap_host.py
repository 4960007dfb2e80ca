"""Which outputs of the norm and its gradient may lie where: refused on the host, before anything is enqueued.  Calls that
overlap nothing are ended by another mistake, looked for later, so that none is enqueued here."""
import random


F32, BF16 = 0, 1


def _lib():
    import fine_grained_blockwise_amd as fgb
    return fgb.lib()


def forward(**kw):
    """(status, message) of a call whose rstd is missing."""
    L = _lib()
    v = dict(x=0x100000, xd=BF16, rows=4, cols=256, ldx=256, r=0x200000, rd=F32, ldr=256, w=0x300000, wd=BF16, h=0x400000,
             ldh=256, rstd=None, q=0x600000, s=0x700000, y=0x800000, yd=BF16, ldy=256)
    v.update(kw)
    rc = L.rmsnorm_quant(v["x"], v["xd"], v["rows"], v["cols"], v["ldx"], v["r"], v["rd"], v["ldr"], v["w"], v["wd"], 1e-6,
                         128, v["h"], v["ldh"], v["rstd"], v["q"], v["s"], v["y"], v["yd"], v["ldy"], None)
    return rc, L.fgb_last_error().decode()


def backward(**kw):
    """... whose workspace is misaligned."""
    L = _lib()
    v = dict(dy=0x100000, dd=BF16, rows=4, cols=256, lddy=256, h=0x200000, hd=F32, ldh=256, w=0x300000, wd=BF16,
             rstd=0x400000, dh=0x500000, lddh=256, dx=0x600000, lddx=256, dw=0x700000, ws=0x800004)
    v.update(kw)
    rc = L.rmsnorm_backward(v["dy"], v["dd"], v["rows"], v["cols"], v["lddy"], v["h"], v["hd"], v["ldh"], v["w"], v["wd"],
                            v["rstd"], v["dh"], v["lddh"], v["dx"], v["lddx"], v["dw"], v["ws"], 1 << 30, None)
    return rc, L.fgb_last_error().decode()


def over(got, what):
    return got[0] == 1 and "lies over" in got[1] and what in got[1]


def test_forward():
    free = lambda **kw: "rstd null" in forward(**kw)[1]  # noqa: E731
    assert free() and free(q=None, s=None) and free(y=None)
    # the very same rows
    assert free(h=0x200000) and free(rd=BF16, h=0x100000) and free(y=0x100000) and free(r=0x100000, rd=BF16, h=0x100000)
    assert free(yd=F32, y=0x200000)
    # of another type, a row further, half a row on, with another stride
    assert over(forward(h=0x100000), "h lies over x") and over(forward(yd=F32, y=0x100000), "y lies over x")
    assert over(forward(h=0x200400), "h lies over residual") and over(forward(h=0x200010), "h lies over residual")
    assert over(forward(h=0x1FFC10), "residual") and over(forward(h=0x200000, ldh=260), "h lies over residual")
    assert over(forward(rows=4, h=0x200FF0), "residual") and free(h=0x201000) and free(h=0x1FF000)
    # single rows have no stride to differ in
    assert free(rows=1, h=0x200000, ldh=512) and over(forward(rows=1, h=0x200010), "residual")
    # every output over the weight, the other outputs and the inputs
    for k in ("h", "y", "q", "s"):
        assert over(forward(**{k: 0x300000}), f"{k} lies over weight"), k
        for other, at in (("h", 0x400000), ("y", 0x800000), ("q", 0x600000), ("s", 0x700000)):
            if other != k:
                got = forward(**{k: at})
                assert over(got, k) and over(got, other), (k, other)
    assert over(forward(q=0x100000), "q lies over x") and over(forward(s=0x200200), "s lies over residual")
    for at, what in ((0x100004, "x"), (0x200004, "residual"), (0x300004, "weight"), (0x400004, "h"), (0x600004, "q"),
                     (0x700004, "s"), (0x800004, "y")):
        assert over(forward(rstd=at), what)
    # without a residual h is not used
    assert free(r=None, h=0x100000)
    # columns of one wide buffer, side by side
    assert free(ldx=1024, ldh=512, ldr=512, x=0x100000, rd=F32, r=0x100200, h=0x100200)
    assert free(ldx=1024, ldh=512, x=0x100000, h=0x100200) and over(forward(ldx=1024, ldh=512, x=0x100000, h=0x1001F0), "x")
    assert over(forward(ldx=1024, ldh=512, x=0x100000, h=0x100410), "x") and free(ldx=1024, ldh=512, h=0x100400)


def test_backward():
    free = lambda **kw: "16-byte aligned" in backward(**kw)[1] and "lies" not in backward(**kw)[1]  # noqa: E731
    assert free() and free(dh=None)
    assert free(dx=0x500000) and free(dx=0x200000) and free(dd=F32, dx=0x100000)
    assert over(backward(dx=0x100000), "dx lies over dy") and over(backward(dx=0x500010), "dx lies over dh")
    assert over(backward(dx=0x200400), "dx lies over h") and over(backward(dx=0x500000, lddx=260), "dh")
    assert over(backward(dx=0x300000), "weight") and over(backward(dx=0x3FF010), "rstd") and over(backward(dx=0x700000), "dweight")
    for at, what in ((0x100000, "dy"), (0x200000, "h"), (0x300000, "weight"), (0x400000, "rstd"), (0x500000, "dh"),
                     (0x600000, "dx"), (0x700000, "dweight")):
        assert over(backward(ws=at), f"workspace lies over {what}"), what
    # nothing is written to dx without rows; the workspace still has to be apart
    assert over(backward(rows=0, dx=None, dy=None, h=None, dh=None, rstd=None, ws=0x700000), "dweight")


def bytes_of(p, rows, n, ld):
    return {p + i * ld + k for i in range(rows) for k in range(0, n, 16)}  # (all are multiples of 16)


def test_every_lie_against_the_bytes_themselves():
    rng = random.Random(0)
    seen = [0, 0]
    for _ in range(4000):
        rows = rng.choice([1, 2, 3, 5, 9])
        cols = rng.choice([32, 64, 96])
        xd, rd = rng.choice([F32, BF16]), rng.choice([F32, BF16])
        xs, rs = (2 if xd else 4), (2 if rd else 4)
        ldx = cols + rng.choice([0, 0, 8, 32, 64, 2 * cols])
        ldh = ldx * xs // rs if rng.random() < 0.6 and ldx * xs // rs >= cols else cols + rng.choice([0, 8, 32, 160])
        x = 0x100000
        h = x + 16 * rng.randint(-120, 120)
        a, b = bytes_of(x, rows, cols * xs, ldx * xs), bytes_of(h, rows, cols * rs, ldh * rs)
        same = x == h and xs == rs and (ldx == ldh or rows == 1)
        want = bool(a & b) and not same
        got = forward(x=x, xd=xd, rows=rows, cols=cols, ldx=ldx, rd=rd, ldr=cols, h=h, ldh=ldh, q=None, s=None)
        assert over(got, "h lies over x") == want and ("rstd null" in got[1]) == (not want), (rows, cols, xd, rd, ldx, ldh, h - x)
        seen[want] += 1
    assert min(seen) > 500


def test_many_rows_of_one_buffer_take_no_time():
    """Rows side by side in one buffer are told apart at once, whatever their number."""
    import time
    t = time.perf_counter()
    for _ in range(20):
        assert "rstd null" in forward(rows=1 << 22, x=1 << 44, ldx=8192, h=(1 << 44) + 0x400, ldh=4096, r=1 << 52, ldr=256,
                                      q=1 << 55, s=1 << 56, y=1 << 57)[1]
    assert time.perf_counter() - t < 1.0
