// The joining of block_attention.cu's parts through a window, included by it in the
// place of its own (inside its namespace).  Blocks are long here: without a prefix nearly every
// row is one worker's and already written, and only the items that workers left
// unfinished (Partials::split) are looked at, a block's warps taking 64 rows of one;
// looking at every row took 97 us for the 45,000 rows of 32 heads of four prompts, this
// takes 26.  The rest, and what is added up, is as there.
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32, 4)
attention_join_kernel(const __grid_constant__ AttentionArgs a, const Partials parts, const int per) {
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const dspark_kv_cache &c = a.cache;
    const int D = c.head_dim, group = a.n_q_heads / c.n_kv_heads, Hq = a.n_q_heads;
    int b = blockIdx.x;
    Request q = load_request(a, b);
    const int prefix_m = prefix_rows(a) * group;
    const int prefix_tiles = prefix_tiles_of(a, *parts.prefix_low);
    // without a prefix only items that a worker left unfinished are joined, in steps of kUnit rows a block
    constexpr int kUnit = 64, kUnits = plan::kTileRows / kUnit;
    const bool listed = prefix_tiles == 0;
    if (q.n == 0 && !listed) return;
    // the line: units of the prefix by class, of all pairs, of all (the last request's end)
    int64_t prefix[2], pairs, total;
    {
        const int last = a.rows.B - 1;
        const Request z = load_request(a, last);
        int64_t end[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            prefix[k] = plan::head_units(k, prefix_m, prefix_tiles) * c.n_kv_heads;
            end[k] = prefix[k] + parts.unit0[k][last] +
                     (z.len_ok && z.n > 0
                          ? plan::head_units(k, z.n * group, own_tiles(a, z.n, z.len, group)) * c.n_kv_heads
                          : 0);
        }
        pairs = end[0];
        total = end[0] + end[1];
    }
    const int64_t all = (int64_t)a.rows.n_rows * Hq;
    auto bad_row = [&](int64_t place) {
        T *out = static_cast<T *>(a.out) + place * D;
        if (lane * 4 < D) *reinterpret_cast<uint2 *>(out + lane * 4) = make_uint2(0x7fff7fffu, 0x7fff7fffu);
        if (lane == 0 && a.lse) a.lse[place] = __int_as_float(0x7fffffff);
    };
    if (listed && blockIdx.y == 0 && !q.len_ok)
        for (int i = warp; i < q.n * Hq; i += kJoinWarps) bad_row(q.first * Hq + i);
    // this lane's item (0 the prefix's, 1 the request's own) and its place among the item's workers
    const int side = lane >> 4, at = lane & 15;
    int64_t own0, own1;
    int own_m, m_of, rows, tiles;
    auto of_request = [&]() {
        own0 = parts.unit0[0][b] + prefix[0], own1 = parts.unit0[1][b] + prefix[1];
        own_m = q.n * group;
        m_of = side ? 0 : (int)q.first * group, rows = side ? own_m : prefix_m;
        tiles = side ? own_tiles(a, q.n, q.len, group) : prefix_tiles;
    };
    if (!listed) of_request();
    const int chunks = listed ? 0 : (own_m + per - 1) / per;
    const int from = listed ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.y * kJoinWarps + warp;
    const int step = listed ? gridDim.x * gridDim.y : gridDim.y * kJoinWarps;
    const int jobs = listed ? 3 * kCtas * kUnits : c.n_kv_heads * chunks;
    for (int i = from; i < jobs; i += step) {
        int h = 0, m0, m1, every = 1;
        if (listed) {
            const int4 record = parts.split[i / kUnits];
            const int first = i % kUnits * kUnit;
            if (record.x < 0 || first >= record.w) continue;
            b = record.x;
            q = load_request(a, b);
            of_request();
            h = record.y;
            m0 = record.z + first + warp;
            m1 = record.z + min(first + kUnit, record.w);
            every = kJoinWarps;
        } else {
            h = i / chunks;
            m0 = (i - h * chunks) * per;
            m1 = min(m0 + per, own_m);
        }
        int item = -1;             // the row tile that is looked at
        bool has = false, first = false, more = false, done = false;
        int64_t part0 = 0;
        // the lane's part of the item, when its worker (the `turn`-th 16 of them) has one
        auto look = [&](int turn) {
            const int cls = plan::class_of(plan::tile_rows(rows, item));
            const int64_t start = (!side ? 0 : cls == plan::kPair ? own0 : own1) + (cls == plan::kPair ? 0 : pairs) +
                                  h * plan::head_units(cls, rows, tiles) +
                                  (cls == plan::kPair ? item * plan::item_total(cls, tiles) : 0);
            const int64_t end = start + plan::item_total(cls, tiles);
            const int v0 = plan::worker_of(cls, start + plan::item_units(cls), pairs, total, kCtas), v = v0 + turn * 16 + at;
            const int workers = cls == plan::kPair ? kCtas : 2 * kCtas;
            has = first = false;
            bool go_on = false, alone = false;
            if (tiles > 0 && v < workers) {
                const int64_t from = plan::worker_begin(cls, v, pairs, total, kCtas);
                const int64_t to = plan::worker_begin(cls, v + 1, pairs, total, kCtas);
                const int t = plan::first_tile(cls, to, start, tiles);
                first = v == v0;
                has = first || (from < end && plan::first_tile(cls, from, start, tiles) < t);
                go_on = at == 15 && to < end && v + 1 < workers;
                alone = first && t == tiles;
            }
            part0 = first ? (side ? all : 0)
                          : 2 * all + (cls == plan::kPair ? 0 : (int64_t)kCtas * plan::kTileRows) +
                                (int64_t)v * (cls == plan::kPair ? plan::kTileRows : plan::kHalfRows);
            more = __any_sync(0xffffffffu, go_on);
            if (turn == 0) done = __any_sync(0xffffffffu, side && alone && prefix_tiles == 0);
        };
        for (int m = m0; m < m1; m += every) {
            const int blk = m / group;
            const int64_t place = (q.first + blk) * Hq + h * group + (m - blk * group);
            T *out = static_cast<T *>(a.out) + place * D;
            if (!q.len_ok) {
                bad_row(place);
                continue;
            }
            const int mt = m_of + m, now = mt / plan::kTileRows;
            const bool other = __any_sync(0xffffffffu, now != item);
            item = now;
            if (other) look(0);
            if (done) continue;
            float top = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
            int turn = 0;
            while (true) {
                const int64_t part = part0 + (first ? place : mt - now * plan::kTileRows);
                float2 st = make_float2(-INFINITY, 0.f);
                if (has && mt < rows) st = parts.stats[part];
                const bool saw = !(st.x == -INFINITY && st.y == 0.f);
                float t = fmaxf(top, st.x);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                const float keep = top == -INFINITY && l == 0.f ? 0.f : scale_down(1.f, top - t);
                const float f = saw ? scale_down(1.f, st.x - t) : 0.f;
                float s = saw ? scale_down(st.y, st.x - t) : 0.f;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                l = (top == -INFINITY && l == 0.f ? 0.f : scale_down(l, top - t)) + s;
                top = t;
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] *= keep;
                unsigned left = __ballot_sync(0xffffffffu, saw);
                while (left) {
                    // two parts at a time
                    const int x = __ffs(left) - 1;
                    left &= left - 1;
                    const int y = left ? __ffs(left) - 1 : x;
                    const float fx = __shfl_sync(0xffffffffu, f, x), fy = left ? __shfl_sync(0xffffffffu, f, y) : 0.f;
                    const int64_t px = __shfl_sync(0xffffffffu, part, x), py = __shfl_sync(0xffffffffu, part, y);
                    if (lane * 4 < D) {
                        const float4 ox = *reinterpret_cast<const float4 *>(parts.o + px * D + lane * 4);
                        const float4 oy = left ? *reinterpret_cast<const float4 *>(parts.o + py * D + lane * 4)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
                        acc[0] += ox.x * fx + oy.x * fy, acc[1] += ox.y * fx + oy.y * fy;
                        acc[2] += ox.z * fx + oy.z * fy, acc[3] += ox.w * fx + oy.w * fy;
                    }
                    left &= left - 1;   // (none left: stays 0)
                }
                if (!more) break;
                look(++turn);
            }
            if (turn > 0) item = -1;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (lane * 4 < D) {
                uint2 v;
                v.x = float_to_pair<T>(acc[0] * inv, acc[1] * inv);
                v.y = float_to_pair<T>(acc[2] * inv, acc[3] * inv);
                *reinterpret_cast<uint2 *>(out + lane * 4) = v;
            }
            if (lane == 0 && a.lse) a.lse[place] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
        }
    }
}
