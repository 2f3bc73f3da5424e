"""Which way a call's sizes take in the passes around attention, restated from the launch code: tests assert that
their cases reach the way that they are meant for."""


def tensor_core_prefix(R, Hq, Hkv, d, blocks):
    """Whether a shared prefix of a table of so many blocks goes to the tensor-core kernel."""
    rows = R * Hq // Hkv
    sets = -(-rows // 16) * Hkv
    if d == 64:
        return sets >= 512 or (sets >= 16 and sets * blocks >= (3000 if blocks >= 60 else 8000))
    if rows < 16:
        return False
    return (Hkv == 1 and sets <= 4 and 16 <= blocks <= 400) or 60 <= blocks <= 128 or \
        (sets >= 4 and sets * blocks >= 2000) or sets >= 256


def piece_blocks(sets, blocks):
    """Cache blocks of a piece."""
    pieces = min(64, max(1, -(-148 * 12 // sets)))
    c = max(8, -(-blocks // pieces))
    return -(-c // 4) * 4


def shared_workspace(R, Hq, Hkv, d, blocks, max_blocks, tensor_cores):
    """Bytes of the shared call's workspace, on either way."""
    align = lambda n: -(-n // 256) * 256
    rows = R * Hq // Hkv
    own = -(-max_blocks // piece_blocks(R * Hkv, max_blocks))
    tiles = pre = 0
    if tensor_cores:
        items = -(-R // (2 * (128 // (Hq // Hkv)))) * Hkv
        tiles = items * (-(-148 // items) + 1) * 256
    else:
        pre = -(-blocks // piece_blocks(-(-rows // 16) * Hkv, blocks))
    results = R * Hq * (own + pre)
    return align(results * d * 4) + align(results * 4) + tiles * (d + 1) * 4


def rope_shape(tokens, heads, d):
    """(token groups of a CTA, rows of a warp) of the norm and rotation."""
    groups = -(-tokens // (32 // (d // 16)))
    warps = 8
    while warps > 1 and heads < 10 * warps and groups * (warps // 2) >= 8 * 4 * 148:
        warps //= 2
    return 8 // warps, -(-heads // warps)


def evict_moves_itself(max_blocks, keep):
    """Whether the selecting CTAs move the rows."""
    M = 16 * max_blocks
    return M <= 40960 and max(0, min(keep, M - keep)) <= 512
