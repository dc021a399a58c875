// The pass of linear_attention.h: the body of la_pass, and of the function that the
// kernels of two passes call.  (Included twice instead of called by both: through
// the function, the compiler's registers for la_pass come out up to 2.5 % slower: a
// gradient over 4 x 8192, 16 heads of 128, 768 us and 755, over 4 x 2048 in float32 575
// and 560; prompts the same.)  In scope: p, m, and the number of
// blocks and this block's index, `blocks` and `index`.
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int kStateParts = !kBf16 ? 1 : kDot != 0 ? 3 : 2;  // of the state as an operand
  constexpr bool kExact = !kBf16 || kDot != 0;             // float32 results depend on the scores
  constexpr int NR = C / 16, NK = C / 32, NM = DA / 16, TB = 64 * NT;
  using Shared = Lds<T, C, DA, NT, kHeads, kOut, kDot>;
  constexpr int PP = Shared::PP, kHeadP = Shared::PR * PP;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;

  static_assert(kHeads == 1 || (NT == 2 && kDot == 0), "two heads of up to 64 columns");
  static_assert(sizeof(Decay<C>) % sizeof(f32x4) == 0 && offsetof(Shared, d) % sizeof(f32x4) == 0 &&
                    offsetof(Shared, p) % sizeof(f32x4) == 0 &&
                    (kDot != 1 || offsetof(Shared, cols) % sizeof(f32x4) == 0),
                "four values are read and written at once");
  const uint32_t block = logical_block(blocks, index);
  const uint32_t groups = static_cast<uint32_t>(p.heads) / kHeads;
  const int64_t slot = block / groups;
  const int h = static_cast<int>(block % groups) * kHeads;
  const int hw = kHeads == 2 ? wave >> 1 : 0;              // this wavefront's head is h + hw
  Place at = place_of(p.grid, slot);
  if (!at.ok) {
    if constexpr (kDot == 2) {
      if (p.head_part && tid == 0) p.head_part[block] = 0.0f;
    }
    return;
  }
  // a state-only pass has nothing to do for the segment that no other follows
  const bool last_seg = kRev ? at.local == 0 : at.local == at.count - 1;
  if (!kOut && last_seg) return;
  bool whole = true;                       // nothing of the segment is out of reach
  if constexpr (!kOut) {
    if (at.len >= kReachFrom) {
      __shared__ Reach look[kHeads];
      int n = 0;
#pragma unroll
      for (int hh = 0; hh < kHeads; ++hh)
        n = max(n, reach<kRev>(look[hh], p.g + at.start * p.g_row + h + hh, p.g_row,
                               static_cast<int>(at.len), tid));
      const int64_t beyond = kRev ? max(at.len - int64_t(n + C - 1) / C * C, int64_t(0))
                                  : (at.len - n) / C * C;           // whole chunks
      whole = beyond == 0;
      if (!kRev) at.start += beyond;
      at.len -= beyond;
    }
  }

  // columns of this wavefront: with two tiles, lane group g4's rows 4 g4 + r of
  // both are the eight consecutive columns 8 g4 + 4 t + r (16-byte stores)
  constexpr int kStep = NT == 2 ? 8 : 4;
  const int c_wave = 16 * NT * wave;
  const int c_head = c_wave - 64 * hw;                     // of its head's columns
  auto col_of = [&](int t, int c) { return c_head + kStep * (c >> 2) + 4 * t + (c & 3); };

  const int64_t sh = (at.seq * p.heads + h + hw) * (int64_t(p.dA) * p.dB);        // per sequence
  const int64_t wh = (slot * p.heads + h + hw) * (int64_t(p.dA) * p.dB);          // per segment

  // the state: rows 16 mt + 4 g4 + r of dA, column col_of(t, l16)
  auto row_of = [&](int mt, int r) { return 16 * mt + 4 * g4 + r; };
  f32x4 s[NM][NT];
  {
    const float* init = !kOut ? nullptr
                        : p.seg_states ? p.seg_states + wh
                        : p.init ? p.init + sh : nullptr;
#pragma unroll
    for (int mt = 0; mt < NM; ++mt)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = col_of(t, l16);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int a = row_of(mt, r);
          s[mt][t][r] = init && a < p.dA && c < p.dB ? init[a * p.sA + c * p.sB] : 0.0f;
        }
      }
  }

  const int chunks = static_cast<int>((at.len + C - 1) / C);
  const float scale = p.scale;
  // A chunk's tiles on their way from memory.  The loads run one chunk ahead of
  // their use, or two, with a second set of registers where state, results and
  // both sets leave room for two blocks on a compute unit (256 registers).  The
  // log decays run two ahead: a chunk's factors are made while the one before is
  // worked on.
  struct Stage {
    Tile<T, C, DA> x, y;
    Tile<T, C, TB, kHeads> z;
    Tile<T, C, TB> e;
  };
  constexpr int kStage = (kOut ? Tile<T, C, DA>::kPieces : 0) * 4 + Tile<T, C, DA>::kPieces * 4 +
                         Tile<T, C, TB>::kPieces * 4 * (kDot == 1 ? 2 : 1);
  constexpr int kHeld = NM * NT * 4 + (kOut ? NR * NT * 4 : 0) + (kDot == 2 ? NR * NT * 4 : 0);
  constexpr int kSets = kHeld + 2 * kStage <= (kOut ? 112 : 128) ? 2 : 1;
  constexpr bool kLate = kOut && kHeld + kStage > 100;
  Stage sets[kSets];
  // Tokens of the it-th chunk worked on, and the pointers to the next chunk to load.
  const int len = static_cast<int>(at.len);
  auto tokens_of = [&](int it) { return min(len - (kRev ? chunks - 1 - it : it) * C, C); };
  const int64_t first = at.start + (kRev && chunks > 0 ? int64_t(chunks - 1) * C : 0);
  auto begin = [&](const View& v, int size) {
    return static_cast<const T*>(v.p) + first * v.row + int64_t(h / v.div) * size;
  };
  const T* X = kOut ? begin(p.x, p.dA) : nullptr;
  const T* Y = begin(p.y, p.dA);
  const T* Z = begin(p.z, p.dB);
  const T* E = kDot == 1 ? begin(p.e, p.dB) : nullptr;
  // (the wavefronts that make the decays load them: one for each head)
  const float* G = p.g + (p.g_row ? first * p.g_row : 0) + h + (kHeads == 2 ? wave & 1 : 0);
  constexpr int kAhead = kRev ? -C : C;                     // tokens from chunk to chunk
  const uint32_t x_row = static_cast<uint32_t>(p.x.row), y_row = static_cast<uint32_t>(p.y.row);
  const uint32_t z_row = static_cast<uint32_t>(p.z.row), e_row = static_cast<uint32_t>(p.e.row);
  const uint32_t g_row = static_cast<uint32_t>(p.g_row);
  // Past the last chunk these load it again (unused).
  auto fetch_g = [&](int it) __attribute__((always_inline)) {
    const float g = G[static_cast<uint32_t>(min(lane, tokens_of(it) - 1)) * g_row];
    if (it + 1 < chunks) G += kAhead * static_cast<int64_t>(g_row);
    return g;
  };
  auto fetch = [&](Stage& f, int it) __attribute__((always_inline)) {
    const int n = tokens_of(it);
    const int64_t next = it + 1 < chunks ? kAhead : 0;
    if constexpr (kOut) {
      f.x.fetch(X, x_row, n, p.dA);
      X += next * x_row;
    }
    f.y.fetch(Y, y_row, n, p.dA);
    Y += next * y_row;
    f.z.fetch(Z, z_row, n, p.dB);
    Z += next * z_row;
    if constexpr (kDot == 1) {
      f.e.fetch(E, e_row, n, p.dB);
      E += next * e_row;
    }
  };
  // The chunk being worked on: where its output, and what is dotted with it, begin.
  const uint32_t o_row = static_cast<uint32_t>(p.heads) * p.dB;
  V* out = kOut ? static_cast<V*>(p.out) + first * o_row + int64_t(h) * p.dB : nullptr;
  const T* dotted = kDot == 2 ? begin(p.e, p.dB) : nullptr;
  float* u_at = kDot != 0 ? p.u + first * p.heads + h : nullptr;
  float* dg_at = kDot == 2 && p.dg ? p.dg + first * p.heads + h : nullptr;

  constexpr int kDumpSize = DA * TB;
  const int64_t chunk0 = slot * p.chunks_per_slot + (p.by_token ? at.start / C : 0);
  const int64_t dump0 = slot * p.dumps_per_slot + (p.by_token ? at.start / (C * kStride<C>) : 0);
  // The scores' second parts: those of tile (rt, ct) lie in tile (ct, rt) of p, which the
  // mask leaves empty, those of the diagonal below the rest.
  auto rest_at = [&](int rt, int ct) {
    return ((ct == rt ? C : 16 * ct) + l16) * PP + 16 * rt + 4 * g4;
  };
  float edge = 0.0f, head_sum = 0.0f;      // dg's are wavefront 0's
  double decay_sum = 0.0;
  float g_next = 0.0f;                     // log decays of the next chunk

  auto step = [&](int it, Stage& f) __attribute__((always_inline)) {
    const int ck = kRev ? chunks - 1 - it : it;
    const int n = tokens_of(it);
    const Decay<C>& d = m.d[it & 1][hw];
    if constexpr (kOut) f.x.stash(m.x, n, p.dA);
    f.y.stash(m.y, n, p.dA);
    f.z.stash(m.z, n, p.dB);
    if constexpr (kDot == 1) f.e.stash(m.e, n, p.dB);
    block_sync();
    const float g_after = fetch_g(min(it + 2, chunks - 1));
    if constexpr (!kLate) fetch(f, min(it + kSets, chunks - 1));
    const int back = (chunks - 1 - ck) % kStride<C>;
    float* dump = nullptr;
    if constexpr (kDot != 0) {
      if (back == 0)
        dump = p.dumps + ((dump0 + (chunks - 1 - ck) / kStride<C>) * p.heads + h) * int64_t(kDumpSize) +
               tid * 4;
    }
    // (dk: the first half of the state that dq left there, loaded before the products
    // that stand between, into the registers of the tiles now in LDS)
    constexpr int kHalf = kDot == 2 ? NM * NT / 2 : 1;
    f32x4 left[kHalf];
    if constexpr (kDot == 2) {
      if (dump) {
#pragma unroll
        for (int u = 0; u < kHalf; ++u) left[u] = *reinterpret_cast<const f32x4*>(dump + u * (kThreads * 4));
      }
    }
    if constexpr (kDot == 1) {
      if (dump) {
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            *reinterpret_cast<f32x4*>(dump + (mt * NT + t) * (kThreads * 4)) = s[mt][t];
      }
    }
    // the tensor that the carried part is dotted with, and u: used further on
    f32x4 ev[kDot == 2 ? NR : 1][NT];
    float uv = 0.0f, qs = 0.0f;
    if constexpr (kDot == 2) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t i = min(16 * r + l16, n - 1), c = min(col_of(t, 4 * g4), p.dB - 4);
          T raw[4];
          __builtin_memcpy(raw, dotted + (i * e_row + c), sizeof(raw));
#pragma unroll
          for (int q = 0; q < 4; ++q) ev[r][t][q] = to_float(raw[q]);
        }
      uv = u_at[static_cast<uint32_t>(min(lane, n - 1) * p.heads)];
      const f32x4 q = *reinterpret_cast<const f32x4*>(p.q_sums + ((chunk0 + ck) * p.heads + h) * 4);
      qs = (q[0] + q[1]) + (q[2] + q[3]);
    }

    f32x4 acc[NR][NT];
    if constexpr (kOut) {
      // the C x C products of this wavefront's part: tiles (rows of x, rows of
      // y), each result a lane's column i (row of x) and four rows j of y
      constexpr int kWaveTiles = NR == 4 ? 4 : 1;
      const int rt = NR == 4 ? wave : wave >> 1;
      const int i = 16 * rt + l16;
      float row_sum = 0.0f;
      // All of a row tile's products are formed, also those that the mask then
      // drops: without branches between them the loads and products of one hide
      // the latency of the others.
      f32x4 as[kWaveTiles], bs[kDot == 1 ? kWaveTiles : 1];
      {
        Frag<T> xf[DA / 32];
#pragma unroll
        for (int k = 0; k < DA / 32; ++k) xf[k] = frag_row<DA>(m.x, i, 32 * k + 4 * g4);
#pragma unroll
        for (int u = 0; u < kWaveTiles; ++u) {
          const int ct = NR == 4 ? u : wave & 1;
          as[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < DA / 32; ++k)
            mma(as[u], frag_row<DA>(m.y, 16 * ct + l16, 32 * k + 4 * g4), xf[k]);
        }
      }
      if constexpr (kDot == 1) {
        Frag<T> ef[TB / 32];
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) ef[k] = frag_row<TB>(m.e, i, 32 * k + 4 * g4);
#pragma unroll
        for (int u = 0; u < kWaveTiles; ++u) {
          const int ct = NR == 4 ? u : wave & 1;
          bs[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < TB / 32; ++k)
            mma(bs[u], frag_row<TB>(m.z, 16 * ct + l16, 32 * k + 4 * g4), ef[k]);
        }
      }
#pragma unroll
      for (int hh = 0; hh < kHeads; ++hh) {
        const Decay<C>& dh = m.d[it & 1][hh];
        T* const ph = m.p + hh * kHeadP;
        const float gi = dh.hi[i], gil = dh.lo[i];
#pragma unroll
        for (int u = 0; u < kWaveTiles; ++u) {
          const int ct = NR == 4 ? u : wave & 1;
          const bool live = kRev ? ct >= rt : ct <= rt;
          const int j0 = 16 * ct + 4 * g4;
          if (live) {
            f32x4 a = as[u], b = bs[kDot == 1 ? u : 0];
            if (ct == rt) {
              const f32x4 gj = *reinterpret_cast<const f32x4*>(&dh.hi[j0]);
              const f32x4 gjl = *reinterpret_cast<const f32x4*>(&dh.lo[j0]);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const bool in = kRev ? j0 + r >= i : j0 + r <= i;
                const float f = kRev ? exp2_diff<kExact>(gj[r], gjl[r], gi, gil) : exp2_diff<kExact>(gi, gil, gj[r], gjl[r]);
                a[r] = in ? a[r] * (scale * f) : 0.0f;
                if constexpr (kDot == 1) b[r] = j0 + r != i ? a[r] * b[r] : 0.0f;
              }
            } else {
              // through the boundary between the 16 tokens and what is nearer to i
              const int edge16 = kRev ? 16 * ct - 1 : 16 * ct + 15;
              const float fi = scale * (kRev ? exp2_diff<kExact>(dh.hi[edge16], dh.lo[edge16], gi, gil)
                                             : exp2_diff<kExact>(gi, gil, dh.hi[edge16], dh.lo[edge16]));
              const f32x4 fj = *reinterpret_cast<const f32x4*>(&dh.fac[j0]);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                a[r] *= fi * fj[r];
                if constexpr (kDot == 1) b[r] *= a[r];
              }
            }
            lds_store4(ph + i * PP + j0, a);
            if constexpr (kBf16) lds_store4_rest(ph + rest_at(rt, ct), a);
            if constexpr (kDot == 1) {
              row_sum += (b[0] + b[1]) + (b[2] + b[3]);
              // sums over this wavefront's 16 rows i, for each of the four j
#pragma unroll
              for (int r = 0; r < 4; ++r) b[r] = row16_sum(b[r]);
              if (l16 == 0) *reinterpret_cast<f32x4*>(&m.cols[8 * rt * (rt + 1) + j0]) = b;
            }
          } else if (!kBf16 && (ct ^ rt) == 1) {
            lds_store4(ph + i * PP + j0, f32x4{0.0f, 0.0f, 0.0f, 0.0f});   // read with its neighbour
          }
        }
      }
      // the wavefronts with the fewest scores prepare the next chunk's decays
      if ((kRev ? wave > 3 - kHeads : wave < kHeads) && it + 1 < chunks)
        decays<C, kRev>(m.d[(it + 1) & 1][wave & (kHeads - 1)], lane < tokens_of(it + 1) ? g_next : 0.0f, scale, lane);
      if constexpr (kDot == 1) {
        row_sum += __shfl_xor(row_sum, 16, 64);
        row_sum += __shfl_xor(row_sum, 32, 64);
        // with two row tiles, each of a row tile's two wavefronts has a part
        if (g4 == 0) m.rows[NR == 4 ? 0 : wave & 1][i] = row_sum;
      }

      // the carried part: x S
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < DA / 32; ++k) {
        Frag<T> part[NT][kStateParts];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = s[2 * k][t][r], v[4 + r] = s[2 * k + 1][t][r];
          split(v, part[t]);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const Frag<T> xf = frag_row<DA>(m.x, 16 * r + l16, 32 * k + 4 * g4);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < kStateParts; ++q) mma(acc[r][t], part[t][q], xf);
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float fe = d.ein[16 * r + l16];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] *= fe;
      }
      if constexpr (kDot != 0) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int i2 = 16 * r + l16;
          float dot = 0.0f;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f32x4 e4;
            if constexpr (kDot == 1) e4 = lds_load4(m.e + tile_at<T, TB>(i2, col_of(t, 4 * g4)));
            else e4 = ev[r][t];       // past n or dB: acc is zero there, of finite values
#pragma unroll
            for (int q = 0; q < 4; ++q) dot = __builtin_fmaf(acc[r][t][q], e4[q], dot);
          }
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (g4 == 0) m.dot[wave][i2] = dot;
        }
      }
      if constexpr (kDot == 2) {
        if (dump) {
          f32x4 right[kHalf];
#pragma unroll
          for (int u = 0; u < kHalf; ++u)
            right[u] = *reinterpret_cast<const f32x4*>(dump + (kHalf + u) * (kThreads * 4));
          float part = 0.0f;
#pragma unroll
          for (int u = 0; u < NM * NT; ++u) {
            const f32x4 q = u < kHalf ? left[u % kHalf] : right[u % kHalf];
#pragma unroll
            for (int r = 0; r < 4; ++r) part = __builtin_fmaf(q[r], s[u / NT][u % NT][r], part);
          }
          part = wave_sum(part);
          if (lane == 0) m.edge[wave] = part;
        }
      }
      block_sync();
    }
    if constexpr (kLate) fetch(f, min(it + 1, chunks - 1));

    // z by columns, for the scores' product and for the state
    Frag<T> zf[NK][NT];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        zf[k][t] = frag_col<TB, kStep>(m.z, 32 * k, c_wave + 4 * t, lane);

    if constexpr (kOut) {
      // whether both of row tile r's tiles 2 k and 2 k + 1 hold scores, or the diagonal's only
      auto both = [](int k, int r) { return kRev ? 2 * k >= r : 2 * k + 1 <= r; };
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (kRev ? k < r / 2 : k > r / 2) continue;
          const T* at_p = m.p + hw * kHeadP + (16 * r + l16) * PP + 32 * k + 4 * g4;
          Frag<T> pf;
          if constexpr (kBf16) {
            pf = both(k, r) ? frag_at(at_p) : half_frag(lds_read8(at_p + 16 * kRev), kRev);
          } else {
            pf = frag_at(at_p);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(acc[r][t], zf[k][t], pf);
        }
      if constexpr (kBf16) {
        const T* rest = m.p + hw * kHeadP;
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if (kRev ? k < r / 2 : k > r / 2) continue;
            const Frag<T> pf = both(k, r) ? frag_of(lds_read8(rest + rest_at(r, 2 * k)),
                                                    lds_read8(rest + rest_at(r, 2 * k + 1)))
                                          : half_frag(lds_read8(rest + rest_at(r, r)), kRev);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma(acc[r][t], zf[k][t], pf);
          }
      }
      // Stores through a descriptor that ends with the chunk's last value: rows and
      // columns past it are dropped by the hardware, so no branch stands around them.
      // (Buffer accesses, too, take any alignment.)
      {
        const buf_t to = make_buf(out, ((n - 1) * o_row + kHeads * p.dB) * static_cast<uint32_t>(sizeof(V)));
        const uint32_t c = col_of(0, 4 * g4);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const uint32_t off = c < static_cast<uint32_t>(p.dB) ? (16 * r + l16) * o_row + hw * p.dB + c : 0x3ffffff0u;
          buf_store<V, NT>(to, off * static_cast<uint32_t>(sizeof(V)), acc[r]);
        }
      }
      if constexpr (kDot == 1) {
        // Each wavefront finishes 16 tokens, lane group g4 with its part of the sums,
        // and without branches, beside the products.
        const int w = NR == 4 ? wave : wave & 1, i2 = 16 * w + l16;
        const int tile = NR == 4 ? g4 : g4 & 1;
        float qd = m.dot[g4][i2];
        const float rows = m.rows[NR == 4 ? 0 : g4 & 1][i2], cols = m.cols[8 * tile * (tile + 1) + i2];
        float u = (g4 < (NR == 4 ? 1 : w + 1) ? rows : 0.0f) - (g4 >= w && g4 < NR ? cols : 0.0f);
        qd += __shfl_xor(qd, 16, 64);
        u += __shfl_xor(u, 16, 64);
        qd += __shfl_xor(qd, 32, 64);
        u += __shfl_xor(u, 32, 64);
        const bool mine = wave < NR;
        const uint32_t heads = static_cast<uint32_t>(p.heads);
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(qd + u), make_buf(u_at, ((n - 1) * heads + 1) * 4),
            g4 == 0 && mine ? static_cast<int>(i2 * heads * 4) : 0x3ffffff0, 0, 0);
        const float sum = row16_sum(mine && i2 < n ? qd : 0.0f);
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(sum), make_buf(p.q_sums + ((chunk0 + ck) * p.heads + h) * 4, 16),
            lane == 0 ? wave * 4 : 0x3ffffff0, 0, 0);
      }
      if constexpr (kDot == 2) {
        if (wave == 0) {
          const bool in = lane < n;
          const int t = min(lane, C - 1);
          const float kd = in ? (m.dot[0][t] + m.dot[1][t]) + (m.dot[2][t] + m.dot[3][t]) : 0.0f;
          const float u = in ? uv : 0.0f;
          const float before = scan_f32(kd), u_before = scan_f32(u);     // up to this token
          const float after = u + (lane_value(u_before, 63) - u_before); // from it on
          // what passes through the whole chunk
          const float through = dump ? d.all * ((m.edge[0] + m.edge[1]) + (m.edge[2] + m.edge[3]))
                                     : edge - lane_value(before, 63);
          const float dg = after + (before - kd) + through;
          edge = through + qs;
          if (in) {
            if (p.dg) dg_at[static_cast<uint32_t>(lane * p.heads)] = dg;
            head_sum += dg;
          }
        }
      }
    }

    if constexpr (kOut) out += kAhead * static_cast<int64_t>(o_row);
    if constexpr (kDot == 2) {
      dotted += kAhead * static_cast<int64_t>(e_row);
      dg_at += kAhead * p.heads;
    }
    if constexpr (kDot != 0) u_at += kAhead * p.heads;

    // The state after the chunk, from three parts of the weighted z (24 bits): the same
    // state whether it is a result or only on its way to the outputs, so that these do not
    // depend on what else the caller asks for.  (Two parts: packed prompts 298 us instead of
    // 309, the long prompt 895 and 927, but the last state errs by 2e-6 of its norm, not 1e-7.)
    if (it + 1 < chunks || !kOut || (last_seg && p.last)) {
      constexpr int kParts = kBf16 ? 3 : 1;
      const float all = d.all;
#pragma unroll
      for (int mt = 0; mt < NM; ++mt)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[mt][t] *= all;
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        Frag<T> part[NT][kParts];
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&d.w[32 * k + 4 * g4]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&d.w[32 * k + 16 + 4 * g4]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
          unpack(zf[k][t], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= w0[e], v[4 + e] *= w1[e];
          split(v, part[t]);
        }
        // (two row tiles at once, so that products into the same registers, which wait
        // for one another, stand apart)
#pragma unroll
        for (int mt = 0; mt < NM; mt += 2) {
          const Frag<T> yf[2] = {frag_col<DA, 4>(m.y, 32 * k, 16 * mt, lane),
                                 frag_col<DA, 4>(m.y, 32 * k, 16 * mt + 16, lane)};
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(s[mt + u][t], yf[u], part[t][q]);
        }
      }
    }
    if constexpr (!kOut) {
      decay_sum += static_cast<double>(d.hi[C - 1]) + d.lo[C - 1];   // the segment's
    }
    if (!kOut && wave < kHeads && it + 1 < chunks)
      decays<C, kRev>(m.d[(it + 1) & 1][wave & (kHeads - 1)], lane < tokens_of(it + 1) ? g_next : 0.0f, scale, lane);
    g_next = g_after;
    block_sync();
  };
  if (chunks > 0) {
    const float g_first = fetch_g(0);
    g_next = fetch_g(min(1, chunks - 1));
    // Each set's first loads are followed by as many stores as later ones (into an
    // empty buffer, dropped): the waits in the loop then leave that many in flight,
    // where for the sake of the first turn they would otherwise drain them.
    auto no_stores = [&](int k) __attribute__((always_inline)) {
      if constexpr (kOut) {
        const buf_t none = make_buf(out, 0);
        const f32x4 zero[NT] = {};
#pragma unroll
        for (int r = 0; r < NR; ++r) buf_store<V, NT>(none, 64 * (NR * k + r), zero);
      }
    };
    fetch(sets[0], 0);
    no_stores(0);
    if constexpr (kSets == 2) {
      fetch(sets[1], min(1, chunks - 1));
      no_stores(1);
    }
    if (wave < kHeads)
      decays<C, kRev>(m.d[0][wave & (kHeads - 1)], lane < tokens_of(0) ? g_first : 0.0f, scale, lane);
  }
  int it = 0;
  if constexpr (kSets == 2) {
    for (; it + 1 < chunks; it += 2) {
      step(it, sets[0]);
      step(it + 1, sets[1]);
    }
    if (it < chunks) step(it, sets[0]);
  } else {
    for (; it < chunks; ++it) step(it, sets[0]);
  }

  if constexpr (kDot == 2) {
    if (p.head_part && wave == 0) {
      head_sum = wave_sum(head_sum);
      if (lane == 0) p.head_part[slot * p.heads + h] = head_sum;
    }
  }
  float* dst = nullptr;
  if constexpr (kOut) {
    if (last_seg && p.last) dst = p.last + sh;
  } else {
    dst = p.seg_out + wh;
    if (lane == 0 && wave % (4 / kHeads) == 0)
      p.seg_decay[slot * p.heads + h + hw] = whole ? exp2_of(decay_sum) : 0.0f;
  }
  if (!dst) return;
#pragma unroll
  for (int mt = 0; mt < NM; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = col_of(t, l16);
      if constexpr (kDot != 0) {                           // (rows consecutive in memory)
        if (row_of(mt, 0) < p.dA && c < p.dB) store4(dst + row_of(mt, 0) + c * p.sB, s[mt][t]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int a = row_of(mt, r);
          if (a < p.dA && c < p.dB) dst[a * p.sA + c * p.sB] = s[mt][t][r];
        }
      }
    }
