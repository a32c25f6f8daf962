"""The group norm's launch plan restated, so that tests can say which form of
the kernels a case takes.  test_operators_cpu.py compares it with the library's
workspace sizes, which follow from the same plan."""
import math

THREADS, MAX_CLUSTER, SMEM_MOST = 256, 8, 200 << 10


def ceil_div(a, b):
    return -(-a // b)


def stream_blocks(run_bytes):
    return {16: 2, 8: 4, 4: 5, 2: 6}[run_bytes]


def vec_of(elem, channels, *views):
    """Channels a thread takes for views given as (pointer, batch stride, pixel stride), strides of single elements 0."""
    for to in (16, 8, 4):
        if channels % (to // elem) == 0 and all(p % to == 0 and b * elem % to == 0 and s * elem % to == 0 for p, b, s in views):
            return to // elem
    return 1


def plan(batch, pixels, channels, groups, elem, vec, backward):
    cpg, runs, run_bytes = channels // groups, channels // vec, vec * elem
    whole = cpg // math.gcd(cpg, vec)

    def scratch(slab, cluster):
        rows, width = THREADS // slab, slab * vec
        n = rows * (width + 1) * 8 + (0 if backward else width * 16)
        if cluster:
            n += width * 16 + width // cpg * 8 if backward else width // cpg * 24
        return ceil_div(n, 16) * 16

    if pixels and whole <= THREADS:
        slab, blocks = whole, 1
        while 2 * slab <= THREADS and slab < runs and (slab * run_bytes < 32 or batch * ceil_div(runs, slab) > 304):
            slab *= 2
        slabs = batch * ceil_div(runs, slab)
        each = lambda: ceil_div(pixels, blocks * (THREADS // slab))
        while blocks < MAX_CLUSTER and ((each() > 2 and 2 * blocks * slabs <= 152) or (each() > 8 and 2 * blocks * slabs <= 304)):
            blocks *= 2
        whole_batch = backward and batch * blocks <= MAX_CLUSTER
        if blocks * slabs <= 304 and each() <= (6 if backward and not whole_batch else 8):
            data = each() * THREADS * vec * elem
            if data <= SMEM_MOST and scratch(slab, True) + data * (2 if backward else 1) <= SMEM_MOST:
                return dict(cluster=True, vec=vec, slab=slab, rows=THREADS // slab, splits=blocks, passes=blocks, unit=cpg,
                            whole_batch=whole_batch, pixels_a_thread=each())
    slab = min(runs, THREADS)
    if runs > THREADS >= whole:
        slab = THREADS // whole * whole
    nslab = ceil_div(runs, slab)
    if whole <= THREADS:
        slab = ceil_div(ceil_div(runs, nslab), whole) * whole
        nslab = ceil_div(runs, slab)
    rows, wave = THREADS // slab, 152 * stream_blocks(run_bytes)
    shares = lambda least: max(1, least, min(wave // (batch * nslab), pixels // (rows * 4)))
    splits, passes = shares(ceil_div(pixels, rows * (128 if backward else 256))), shares(1)
    unit = cpg if not backward and whole <= THREADS else 1
    return dict(cluster=False, vec=vec, slab=slab, rows=rows, splits=splits, passes=passes, unit=unit, whole_batch=False,
                fold=unit == cpg and splits * (slab * vec // cpg) <= 2048, pixels_a_thread=ceil_div(pixels, rows * splits))


def workspace(batch, pixels, channels, groups, elem, backward):
    if batch == 0:
        return 0
    up, need = lambda n: ceil_div(n, 256) * 256, 0
    for vec in (16 // elem, 8 // elem, 4 // elem, 1):
        if channels % vec:
            continue
        p = plan(batch, pixels, channels, groups, elem, vec, backward)
        n = 0 if p["cluster"] else up(batch * p["splits"] * (channels // p["unit"]) * (8 if backward else 16)) + up(batch * groups * 8)
        n += 0 if not backward or p["whole_batch"] else up(batch * channels * 8)
        need = max(need, n)
    return need


def sum_steps(p, batch, pixels, channels, groups, backward):
    """fp32 roundings, at most, that the longest of the plan's sums goes through from a thread's first pixel to the
    group's (or weight's) sum: a thread's pixels, the rows of a block, the splits, the channels of a group, the batch."""
    cpg, per = channels // groups, p["pixels_a_thread"]
    lanes = 1
    while lanes < 32 and 2 * lanes * p["slab"] * p["vec"] <= THREADS:
        lanes *= 2
    rows = ceil_div(p["rows"], lanes) + int(math.log2(lanes))
    join = cpg if cpg <= 8 else ceil_div(cpg, 32) + 5
    if backward:
        thread = per if p["vec"] >= 4 else 16 + ceil_div(per, 16)
        cols = min(32, 1 << max(0, math.ceil(math.log2(cpg))))
        splits = 0 if p["cluster"] else ceil_div(p["splits"], THREADS // cols) + 8
        return thread + rows + (p["splits"] if p["cluster"] else splits) + max(join + 13, batch)
    # joining two moments takes six roundings: the blocks of a cluster in turn, or splits by lanes (at least splits / 16
    # of them where the pass joins them, else the 128 threads of a block)
    if p["cluster"]:
        turns = p["splits"]
    elif p["fold"]:
        turns = min(p["splits"], 16) + 5
    else:
        turns = ceil_div(p["splits"] * (cpg // p["unit"]), 128) + 8
    return per + rows + join + 6 * turns
